// Gated linear recurrence over the grid's tokens in one of the four scan orders, and its backward pass (an
// elementwise-state companion of the selective scan; the pages describe only the latter).  Per sample and channel:
//   a_t = sigmoid(g_t + bias),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  y_t = h_t            (h_0 given or zero)
// Backward, with the adjoint state l_t = dy_t + m_{t+1}, m_t = a_t l_t (behind the last row: m = gradient of h_last):
//   dx_t = (1 - a_t) l_t,  dg_t = l_t (h_{t-1} - x_t) a_t (1 - a_t),  dbias = sum of dg,  dh0 = m_1.
// States, gates and sums are fp32; y, dx and dg are rounded once on the way out.
//
// A run of rows maps the state before it to the state behind it by h -> A h + H.  The sequence is cut into chunks; a
// thread owns a few channels of a chunk and walks its rows, many loads ahead:
//   1. gated_scan_kernel<false>  the chunks' (A, H);
//   2. gated_carry_kernel        the state before every chunk, joined in a fixed order;
//   3. gated_scan_kernel<true>   the rows again from that state, y out.
// Every x and g is read twice (the last-read rows from L2: step 3 starts where step 1 ended), five streams instead of
// the three that cannot be avoided.  One pass with the chunks' pairs handed on between running blocks was built and
// measured too: it moves three, but needs as many instructions as the two row steps together (60 per two values: staging,
// joins, waiting) and leaves the blocks in step, all waiting for the slowest: 700 us for 262,144 rows of 1024 channels,
// where the three steps take 483.
// A sequence of one chunk takes step 3 alone.
#pragma once
#include "common.cuh"
#include "mamba_extras.cuh"   // to_f32, from_f32

#include <type_traits>

namespace mate {

constexpr int kGsState = 8;      // rows per saved state: the backward pass holds so many rows of a channel pair at a time
constexpr int kGsBatch = kGsState;   // rows that a thread loads at a time
constexpr int kGsThreads = 128, kGsBwdThreads = 256;   // 1 KB of a bf16 row per block either way
static_assert(kGsBatch == kGsState, "a state is saved before every batch of rows");
constexpr int kGsMaxChunk = 128;
constexpr int kGsOneChunk = 64;  // sequences up to this length are one chunk
constexpr int kGsCarryHeld = 8;  // pairs that a thread of the carry kernel holds

// The grid rows of the steps s = 0, 1, .. of a recurrence: three nested counters, fastest first.
struct GsOrder {
  FastDiv n0, n1;
  int base, s0, d1, d2;   // first row; row step; further step when the first, the second counter starts again
};

struct GatedScanParams {
  const void *x, *g;       // rows b*n + raster, strides ldx, ldg
  unsigned ldx, ldg;
  const float* bias;       // [D] or null
  const float* h0;         // [B][D] or null
  void* y;                 // forward
  unsigned ldy;
  float* h_last;           // [B][D] or null
  float* states;           // forward: [B][n / kGsState][D] out or null; backward: in
  const void* dy;          // backward
  unsigned lddy;
  const float* dh_last;    // [B][D] or null
  void *dx, *dg;
  unsigned lddx, lddg;
  float* dh0;              // [B][D] or null
  float* dbias_part;       // [chunks][B][D] partial sums, or null
  float2* pair;            // [chunks][B][D] (A, H)
  float* carry;            // [chunks][B][D] state before the chunk (backward: adjoint behind it); null: one chunk
  GsOrder order, back;     // the steps in the recurrence's order, and from the last one back
  FastDiv per, B;          // threads per (sample, chunk), samples
  int D, n, chunk, chunks, states_per;
  unsigned threads;
};

struct GsWalk {
  int row, c0, c1;
  __device__ __forceinline__ GsWalk(const GsOrder& o, unsigned s) {
    const unsigned q = o.n0.div(s), q2 = o.n1.div(q);
    c0 = s - q * o.n0.d;
    c1 = q - q2 * o.n1.d;
    // every step s0, every wrap of the first counter d1 more, every wrap of the second d2 more (mod 2^32 on the way)
    row = static_cast<int>(static_cast<unsigned>(o.base) + s * static_cast<unsigned>(o.s0) +
                           q * static_cast<unsigned>(o.d1) + q2 * static_cast<unsigned>(o.d2));
  }
  // The next U rows; usually the first counter does not start again among them.
  template <int U>
  __device__ __forceinline__ void take(const GsOrder& o, int (&r)[U]) {
    if (c0 + U < static_cast<int>(o.n0.d)) {
#pragma unroll
      for (int j = 0; j < U; ++j) r[j] = row + j * o.s0;
      row += U * o.s0;
      c0 += U;
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        r[j] = row;
        next(o);
      }
    }
  }
  __device__ __forceinline__ void next(const GsOrder& o) {
    row += o.s0;
    if (++c0 == static_cast<int>(o.n0.d)) {
      c0 = 0;
      row += o.d1;
      if (++c1 == static_cast<int>(o.n1.d)) {
        c1 = 0;
        row += o.d2;
      }
    }
  }
};

// The gate's argument, t = -z log2 e.  g and the bias are added first: scaled first, each by itself, the bias would leave
// its own rounding (27 half steps at g = 60, bias = -55) where the two cancel.
constexpr float kGsLog2e = -1.4426950408889634f;
__device__ __forceinline__ float2 gs_arg(float2 g, float2 bias) { return mul_f32x2(add2(g, bias), both(kGsLog2e)); }

// a = sigmoid(z) and 1 - a, each to its own size: with e = 2^t, a = 1 / (1 + e) (0 where that is below the normal numbers),
// and 1 - a is e a where a is above 1/2, the difference where it is not (there e a may be infinity times 0).  The argument's
// three roundings (the sum, the product, the constant) move the smaller of the two by up to 2.2 |z| half steps, the special
// functions add a few.  NaN stays NaN.
__device__ __forceinline__ float2 gs_keep(float2 t, float2* e) {
  *e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
  const float2 d = add2(*e, both(1.f));
  float2 a;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a.y) : "f"(d.y));
  return a;
}
__device__ __forceinline__ void gs_gate(float2 t, float2* a, float2* na) {
  float2 e;
  *a = gs_keep(t, &e);
  const float2 p = mul_f32x2(e, *a), q = fma2(*a, both(-1.f), both(1.f));
  na->x = t.x < 0.f ? p.x : q.x;
  na->y = t.y < 0.f ? p.y : q.y;
}

// What a run of rows leaves of the state before it: the product of its gates, in [0, 1].  Gates above 0 keep an infinite
// state infinite, and one of 0 makes it NaN, however the rows are cut into runs: so a product of gates above 0 that is too
// small for fp32 stays at the smallest number (of a finite state that adds at most 2^-149 |h|, what rounding such a product
// adds, too), and 0 says that a gate was 0.  A NaN gate is in the run's H.
__device__ __forceinline__ float gs_kept(float A, float a) {
  return fmaxf(A * a, fminf(fminf(A, a), __uint_as_float(1u)));
}

// 2 NP consecutive channels as loaded, and as pairs of fp32.
template <typename T_, int NP>
struct GsRaw {
  uint32_t w[NP * sizeof(T_) / 2];
  __device__ __forceinline__ void load(const T_* p) {
    constexpr int bytes = NP * 2 * sizeof(T_);
    if constexpr (bytes == 16) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (bytes == 8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = u.x; w[1] = u.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  }
  __device__ __forceinline__ float2 get(int k) const {
    if constexpr (sizeof(T_) == 2) return bf16_pair(w[k]);
    else return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
  }
};
template <typename T_, int NP>
__device__ __forceinline__ void gs_store(T_* p, const float2 (&v)[NP]) {
  if constexpr (sizeof(T_) == 2) {
    if constexpr (NP == 2)
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
    else
      *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0].x, v[0].y);
  } else {
    if constexpr (NP == 2) *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    else *reinterpret_cast<float2*>(p) = v[0];
  }
}
template <int NP>
__device__ __forceinline__ void gs_load_f32(const float* p, float2 (&v)[NP]) {
#pragma unroll
  for (int k = 0; k < NP; ++k)
    v[k] = p != nullptr ? reinterpret_cast<const float2*>(p)[k] : make_float2(0.f, 0.f);   // may be written later
}

// Row `row` behind p.
template <typename T_>
__device__ __forceinline__ T_* gs_at(T_* p, int row, unsigned ld) {
  return p + static_cast<unsigned long long>(static_cast<unsigned>(row)) * ld;
}

// A = what a batch leaves of A, from the plain products P of its gates.  Where one came out as 0 (gates below 2^-18 on
// average, or one of 0), the batch's gates, steps s, s + 1, .. of `order`, are multiplied again one by one.
template <typename T_, int NP>
__device__ __forceinline__ void gs_keep_batch(float2 (&A)[NP], float2 (&P)[NP], const GsOrder& order, unsigned s, int count,
                                              const T_* g, unsigned ldg, const float2 (&bias)[NP]) {
  float least = P[0].x;
#pragma unroll
  for (int k = 0; k < NP; ++k) least = fminf(least, fminf(P[k].x, P[k].y));
  if (least == 0.f) {
#pragma unroll
    for (int k = 0; k < NP; ++k) P[k] = both(1.f);
    GsWalk w(order, s);
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      GsRaw<T_, NP> gr;
      gr.load(gs_at(g, w.row, ldg));
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        float2 e;
        const float2 a = gs_keep(gs_arg(gr.get(k), bias[k]), &e);
        P[k] = make_float2(gs_kept(P[k].x, a.x), gs_kept(P[k].y, a.y));
      }
      w.next(order);
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) A[k] = make_float2(gs_kept(A[k].x, P[k].x), gs_kept(A[k].y, P[k].y));
}

// Which channels (2 NP from c on) of which chunk a thread takes.
struct GsItem {
  int b, k, c;
  long long bc;   // b * D + c
  template <int NP>
  __device__ __forceinline__ void set(const GatedScanParams& p, unsigned t) {
    const unsigned r = p.per.div(t), q = p.B.div(r);
    c = static_cast<int>(t - r * p.per.d) * 2 * NP;
    b = r - q * p.B.d;
    k = q;
    bc = (long long)b * p.D + c;
  }
};

// Four channels of a chunk per thread.  OUT: y from the state before the chunk (and the states every kGsState rows, the
// last state); else the chunk's pair.  Bound by HBM with eight rows of two tensors in flight per thread: 262,144 rows of
// 1024 bf16 channels take 209 us for the pairs (0.78 of the measured copy rate; 190 before g and the bias were added first,
// 205 before products of gates were kept above 0) and 257 us for y (0.96); more registers for y's step (fewer blocks) cost
// 25%, and guards on every row and its position some 20%.
template <typename T_, bool OUT>
__global__ void __launch_bounds__(kGsThreads, sizeof(T_) == 4 ? 4 : OUT ? 6 : 8) gated_scan_kernel(const GatedScanParams p) {
  constexpr int NP = 2, U = kGsBatch;
  unsigned t = blockIdx.x * blockDim.x + threadIdx.x;
  if (OUT) t = gridDim.x * blockDim.x - 1 - t;   // from the end: the rows that the first step read last
  if (t >= p.threads) return;
  GsItem it;
  it.set<NP>(p, t);
  const int s0 = it.k * p.chunk, rows = min(p.chunk, p.n - s0);
  const float2 one = both(1.f), zero = both(0.f);
  float2 bias[NP], A[NP], h[NP];
  gs_load_f32<NP>(p.bias != nullptr ? p.bias + it.c : nullptr, bias);
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    A[k] = one;
    h[k] = zero;
  }
  if (OUT) {
    // several chunks: the first one's state comes from the carries too, since h_last may be h0
    if (p.chunks > 1) gs_load_f32<NP>(p.carry + (long long)it.k * p.B.d * p.D + it.bc, h);
    else gs_load_f32<NP>(p.h0 != nullptr ? p.h0 + it.bc : nullptr, h);
  }
  const T_* x = static_cast<const T_*>(p.x) + (long long)it.b * p.n * p.ldx + it.c;
  const T_* g = static_cast<const T_*>(p.g) + (long long)it.b * p.n * p.ldg + it.c;
  T_* y = OUT ? static_cast<T_*>(p.y) + (long long)it.b * p.n * p.ldy + it.c : nullptr;
  float* st = OUT && p.states != nullptr
                  ? p.states + ((long long)it.b * p.states_per + s0 / kGsState) * p.D + it.c : nullptr;
  GsWalk w(p.order, s0);
  auto batch = [&](int i, auto all) {   // all U rows are there, or up to the end
    constexpr bool whole = decltype(all)::value;
    int row[U];
    GsRaw<T_, NP> xr[U], gr[U];
    w.take(p.order, row);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (whole || i + j < rows) {
        xr[j].load(gs_at(x, row[j], p.ldx));
        gr[j].load(gs_at(g, row[j], p.ldg));
      }
    if (OUT && st != nullptr) {
#pragma unroll
      for (int k = 0; k < NP; ++k) reinterpret_cast<float2*>(st)[k] = h[k];
      st += p.D;
    }
    float2 P[NP];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (whole || i + j < rows) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          float2 a, na;
          gs_gate(gs_arg(gr[j].get(k), bias[k]), &a, &na);
          h[k] = fma2(a, h[k], mul_f32x2(na, xr[j].get(k)));
          if (!OUT) P[k] = j == 0 ? a : mul_f32x2(P[k], a);
        }
        if (OUT) gs_store<T_, NP>(gs_at(y, row[j], p.ldy), h);
      }
    if (!OUT) gs_keep_batch<T_, NP>(A, P, p.order, s0 + i, whole ? U : rows - i, g, p.ldg, bias);
  };
  int i = 0;
  for (; i + U <= rows; i += U) batch(i, std::true_type{});
  if (i < rows) batch(i, std::false_type{});
  if (OUT) {
    if (p.h_last != nullptr && it.k + 1 == p.chunks)
#pragma unroll
      for (int k = 0; k < NP; ++k) reinterpret_cast<float2*>(p.h_last + it.bc)[k] = h[k];
  } else {
    float4* o = reinterpret_cast<float4*>(p.pair + (long long)it.k * p.B.d * p.D + it.bc);
#pragma unroll
    for (int k = 0; k < NP; ++k) o[k] = make_float4(A[k].x, h[k].x, A[k].y, h[k].y);
  }
}

// The chunks' pairs of the adjoint state, m -> A m + M from the row behind a chunk to the row before it (60 us for 65,536
// rows of 1024 bf16 channels, two streams: 0.68 of the copy rate).
template <typename T_>
__global__ void __launch_bounds__(kGsThreads, sizeof(T_) == 4 ? 4 : 8) gated_adjoint_kernel(const GatedScanParams p) {
  constexpr int NP = 2, U = kGsBatch;
  const unsigned t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= p.threads) return;
  GsItem it;
  it.set<NP>(p, t);
  const int s0 = it.k * p.chunk, rows = min(p.chunk, p.n - s0);
  float2 bias[NP], A[NP], m[NP];
  gs_load_f32<NP>(p.bias != nullptr ? p.bias + it.c : nullptr, bias);
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    A[k] = both(1.f);
    m[k] = both(0.f);
  }
  const T_* g = static_cast<const T_*>(p.g) + (long long)it.b * p.n * p.ldg + it.c;
  const T_* dy = static_cast<const T_*>(p.dy) + (long long)it.b * p.n * p.lddy + it.c;
  GsWalk w(p.back, p.n - s0 - rows);
  auto batch = [&](int i, auto all) {
    constexpr bool whole = decltype(all)::value;
    int row[U];
    GsRaw<T_, NP> gr[U], dr[U];
    w.take(p.back, row);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (whole || i + j < rows) {
        gr[j].load(gs_at(g, row[j], p.ldg));
        dr[j].load(gs_at(dy, row[j], p.lddy));
      }
    float2 P[NP];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (whole || i + j < rows)
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          float2 e;
          const float2 a = gs_keep(gs_arg(gr[j].get(k), bias[k]), &e);
          m[k] = mul_f32x2(a, add2(dr[j].get(k), m[k]));
          P[k] = j == 0 ? a : mul_f32x2(P[k], a);
        }
    gs_keep_batch<T_, NP>(A, P, p.back, p.n - s0 - rows + i, whole ? U : rows - i, g, p.ldg, bias);
  };
  int i = 0;
  for (; i + U <= rows; i += U) batch(i, std::true_type{});
  if (i < rows) batch(i, std::false_type{});
  float4* o = reinterpret_cast<float4*>(p.pair + (long long)it.k * p.B.d * p.D + it.bc);
#pragma unroll
  for (int k = 0; k < NP; ++k) o[k] = make_float4(A[k].x, m[k].x, A[k].y, m[k].y);
}

// carry [chunks][cols] (cols = B D) from the pairs: the start value (null: 0) carried over the chunks, `back`: from the
// last chunk to the first.  A block takes CH columns; each of its SEG threads per column joins a run of chunks, then the
// runs before it in order, then walks its run again.  Latency bounds it, so the runs are as many as give a thread eight
// chunks or so (8 samples of 112 chunks, 512 columns: a scan of 18.6 us with 32 runs, 22.0 with 64, 31.9 with 128).
template <int CH, int SEG>
__global__ void __launch_bounds__(CH * SEG)
    gated_carry_kernel(const float2* __restrict__ pair, const float* __restrict__ start, float* __restrict__ carry,
                       int chunks, int cols, int back) {
  __shared__ float2 s[SEG][CH];
  const int lc = threadIdx.x % CH, seg = threadIdx.x / CH, c = blockIdx.x * CH + lc;
  const int len = (chunks + SEG - 1) / SEG, k0 = min(seg * len, chunks), k1 = min(k0 + len, chunks);
  const bool live = c < cols;
  auto at = [&](int k) { return (long long)(back ? chunks - 1 - k : k) * cols + c; };
  float2 v[kGsCarryHeld];   // the run's first pairs, held for the second walk
  float A = 1.f, H = 0.f;
  if (live) {
#pragma unroll
    for (int j = 0; j < kGsCarryHeld; ++j) v[j] = k0 + j < k1 ? pair[at(k0 + j)] : make_float2(1.f, 0.f);
#pragma unroll
    for (int j = 0; j < kGsCarryHeld; ++j) {
      H = fmaf(v[j].x, H, v[j].y);
      A = gs_kept(A, v[j].x);
    }
#pragma unroll 8
    for (int k = k0 + kGsCarryHeld; k < k1; ++k) {
      const float2 u = pair[at(k)];
      H = fmaf(u.x, H, u.y);
      A = gs_kept(A, u.x);
    }
  }
  s[seg][lc] = make_float2(A, H);
  const float h0 = live && start != nullptr ? start[c] : 0.f;
  __syncthreads();
  if (!live) return;
  float h = h0;
#pragma unroll 8
  for (int q = 0; q < seg; ++q) h = fmaf(s[q][lc].x, h, s[q][lc].y);
#pragma unroll
  for (int j = 0; j < kGsCarryHeld; ++j)
    if (k0 + j < k1) {
      carry[at(k0 + j)] = h;
      h = fmaf(v[j].x, h, v[j].y);
    }
#pragma unroll 8
  for (int k = k0 + kGsCarryHeld; k < k1; ++k) {
    carry[at(k)] = h;
    const float2 u = pair[at(k)];
    h = fmaf(u.x, h, u.y);
  }
}

// Gradients: two channels of a chunk per thread, kGsState rows at a time from the last to the first.  Their states are
// formed again from the saved one, then the adjoint state walks back over them.  148 us for 65,536 rows of 1024 bf16
// channels (five streams and the states: 0.73 of the copy rate), bound by the loads in flight at 128 registers: sixteen
// rows at a time spilled (3.8 times the time), blocks of 128 threads, half a KB of a row each, took 14% longer, 80 registers
// 15%.
template <typename T_>
__global__ void __launch_bounds__(kGsBwdThreads, 2) gated_scan_bwd_kernel(const GatedScanParams p) {
  constexpr int U = kGsState;
  const unsigned t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= p.threads) return;
  GsItem it;
  it.set<1>(p, t);
  const int s0 = it.k * p.chunk, rows = min(p.chunk, p.n - s0);
  float2 bias[1], m[1], db = both(0.f);
  gs_load_f32<1>(p.bias != nullptr ? p.bias + it.c : nullptr, bias);
  if (p.chunks > 1) gs_load_f32<1>(p.carry + (long long)it.k * p.B.d * p.D + it.bc, m);   // dh0 may be dh_last
  else gs_load_f32<1>(p.dh_last != nullptr ? p.dh_last + it.bc : nullptr, m);
  const T_* x = static_cast<const T_*>(p.x) + (long long)it.b * p.n * p.ldx + it.c;
  const T_* g = static_cast<const T_*>(p.g) + (long long)it.b * p.n * p.ldg + it.c;
  const T_* dy = static_cast<const T_*>(p.dy) + (long long)it.b * p.n * p.lddy + it.c;
  T_* dx = static_cast<T_*>(p.dx) + (long long)it.b * p.n * p.lddx + it.c;
  T_* dg = static_cast<T_*>(p.dg) + (long long)it.b * p.n * p.lddg + it.c;
  const float* st = p.states + ((long long)it.b * p.states_per + s0 / kGsState) * p.D + it.c;
  GsWalk w(p.back, p.n - s0 - rows);
  auto batch = [&](int i, auto all) {   // rows i .. i + U - 1 of the chunk (or up to its end), last to first
    constexpr bool whole = decltype(all)::value;
    int row[U];   // from the last one back
    GsRaw<T_, 1> xr[U], gr[U], dr[U];
    const int skip = whole ? 0 : U - (rows - i);   // rows behind the end
    if (whole) {
      w.take(p.back, row);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (j >= skip) {
          row[j] = w.row;
          w.next(p.back);
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (whole || j >= skip) {
        xr[j].load(gs_at(x, row[j], p.ldx));
        gr[j].load(gs_at(g, row[j], p.ldg));
        dr[j].load(gs_at(dy, row[j], p.lddy));
      }
    float2 h = __ldg(reinterpret_cast<const float2*>(st + (long long)(i / U) * p.D));
    float2 a[U], na[U], d[U];   // d: the state before the row, less x
#pragma unroll
    for (int j = U - 1; j >= 0; --j)
      if (whole || j >= skip) {
        const float2 xv = xr[j].get(0);
        gs_gate(gs_arg(gr[j].get(0), bias[0]), &a[j], &na[j]);
        d[j] = fma2(xv, both(-1.f), h);
        h = fma2(a[j], h, mul_f32x2(na[j], xv));
      }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (whole || j >= skip) {
        const float2 l = add2(dr[j].get(0), m[0]);
        const float2 o[1] = {mul_f32x2(na[j], l)};
        m[0] = mul_f32x2(a[j], l);
        const float2 v[1] = {mul_f32x2(mul_f32x2(o[0], d[j]), a[j])};
        gs_store<T_, 1>(gs_at(dx, row[j], p.lddx), o);
        gs_store<T_, 1>(gs_at(dg, row[j], p.lddg), v);
        db = add2(db, v[0]);
      }
  };
  int i = rows / U * U;
  if (i < rows) batch(i, std::false_type{});
  for (i -= U; i >= 0; i -= U) batch(i, std::true_type{});
  if (it.k == 0 && p.dh0 != nullptr) *reinterpret_cast<float2*>(p.dh0 + it.bc) = m[0];
  if (p.dbias_part != nullptr) *reinterpret_cast<float2*>(p.dbias_part + (long long)it.k * p.B.d * p.D + it.bc) = db;
}

}  // namespace mate
