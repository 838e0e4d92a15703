// Gated linear recurrence over the grid's tokens in one of the four scan orders, and its backward pass (an
// elementwise-state companion of the selective scan; the pages describe only the latter).  Per sample and channel:
//   a_t = sigmoid(g_t + bias),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  y_t = h_t            (h_0 given or zero)
// Backward, with the adjoint state l_t = dy_t + m_{t+1}, m_t = a_t l_t (behind the last row: m = gradient of h_last):
//   dx_t = (1 - a_t) l_t,  dg_t = l_t (h_{t-1} - x_t) a_t (1 - a_t),  dbias = sum of dg,  dh0 = m_1.
// States, gates and sums are fp32; y, dx and dg are rounded once on the way out.
//
// One pass over the data.  A tile is a run of rows x 64 channels; a run of rows maps the state before it to the state
// behind it by h -> A h + H, and such pairs (A, H) join in order.  Persistent blocks take tiles by ticket (all
// channels and samples of the first rows, then the next rows).  One warp gathers the next tiles' rows by TMA (four rows
// per instruction, whatever the scan order) into a ring; all eight form the tile's pair, publish it, and find the
// state before the tile from the pairs of the tiles before it in its group of kGsGroup tiles and the state before that
// group, which the last tile of the group before publishes.  (A ninth warp for the loads would leave the others 96
// registers: five warps on one scheduler.)  The joins are the same ones in the same order on every
// run, whoever publishes first, so the result is reproducible.  A ticket only waits for smaller tickets, and a block
// works its tickets off in order, so the smallest unfinished tile can always finish: nothing depends on how many
// blocks run at a time.
#pragma once
#include "common.cuh"
#include "mamba_extras.cuh"   // to_f32, from_f32

namespace mate {

constexpr int kGsChan = 64;            // channels per tile: 32 lanes x 2
constexpr int kGsWarps = 8;
constexpr int kGsThreads = kGsWarps * 32;
constexpr int kGsLoadWarp = 4;         // the first and the last warp have the tile's total to form
constexpr int kGsGroup = 32;           // tiles per group: at most 31 pairs to join behind the group's state
constexpr int kGsShort = 8;            // longest sequence of the short kernel

// Rows per thread and per tile (the forward's `states` hold the state before each tile).  The gates and terms of a
// thread's rows stay in registers between the two halves of the work.
template <typename T_>
constexpr int kGsRun = sizeof(T_) == 2 ? 16 : 8;
template <typename T_>
constexpr int kGsRows = kGsWarps * kGsRun<T_>;
template <typename T_, int NT>
constexpr int kGsStages = NT == 2 ? 3 : 2;

struct GatedScanParams {
  const void *x, *g;       // rows b*n + raster, strides ldx, ldg
  long long ldx, ldg;
  const float* bias;       // [D] or null
  const float* h0;         // [B][D] or null
  void* y;                 // forward
  long long ldy;
  float* h_last;           // [B][D] or null
  float* states;           // forward: [B][tiles][D] out or null; backward: in
  const void* dy;          // backward
  long long lddy;
  const float* dh_last;    // [B][D] or null
  void *dx, *dg;
  long long lddx, lddg;
  float* dh0;              // [B][D] or null
  float* dbias_part;       // [B * tiles][D] partial sums, or null
  unsigned* ticket;        // null: one tile of rows, no joins
  unsigned* abort;         // set when a wait ran out: the blocks leave
  unsigned long long* pair;    // [tiles][B][D] published (A, H) pairs
  unsigned long long* group;   // [groups][B][D] state before a group (low word 0, state in the high word)
  int B, T, H, W, D;
  int n, tiles, cblocks;   // rows of a sample, tiles of rows, tiles of channels
  int order, reverse;
};

constexpr unsigned kGsEmpty = 0xffffffffu;   // low word of what nobody has published yet (the workspace is filled with ones)

// Grid row (of its sample) of step s of the recurrence.
__device__ __forceinline__ int gs_row(const GatedScanParams& p, int s) {
  return scan_to_raster(p.reverse ? p.n - 1 - s : s, p.T, p.H, p.W, p.order);
}

// a = sigmoid(z) and 1 - a, each to full precision, from t = -z log2 e: with e = 2^t, a = 1 / (1 + e) (0 where that is
// below the normal numbers), and 1 - a is e a where a is above 1/2, the difference where it is not (there e a may be
// infinity times 0).  NaN stays NaN.
__device__ __forceinline__ void gs_gate(float2 t, float2* a, float2* na) {
  const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
  const float2 d = add2(e, both(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a->x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a->y) : "f"(d.y));
  const float2 p = mul_f32x2(e, *a), q = fma2(*a, both(-1.f), both(1.f));
  na->x = t.x < 0.f ? p.x : q.x;
  na->y = t.y < 0.f ? p.y : q.y;
}
constexpr float kGsLog2e = -1.4426950408889634f;

// Data and validity travel in one 64-bit word per channel (A below, H above), so publishing needs no fence and reading
// no second look.  A vector access is one access per 64-bit element.
struct GsPair {
  unsigned long long x, y;   // of a thread's two channels
};
__device__ __forceinline__ unsigned long long gs_word(float lo, float hi) { return f2_bits(make_float2(lo, hi)); }
__device__ __forceinline__ void gs_publish(unsigned long long* w, float2 A, float2 H) {
  // the low word may not look empty: a NaN gets the payload that arithmetic gives it
  if (A.x != A.x) A.x = __uint_as_float(0x7fffffffu);
  if (A.y != A.y) A.y = __uint_as_float(0x7fffffffu);
  asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(w), "l"(gs_word(A.x, H.x)), "l"(gs_word(A.y, H.y))
               : "memory");
}
__device__ __forceinline__ GsPair gs_look(const unsigned long long* w) {
  GsPair v;
  asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "l"(w) : "memory");
  return v;
}
__device__ __forceinline__ bool gs_empty(const GsPair& v) {
  return static_cast<unsigned>(v.x) == kGsEmpty || static_cast<unsigned>(v.y) == kGsEmpty;
}
constexpr unsigned kGsMaxPolls = 1u << 20;   // about a second

// Waits until a pair is published; false if the wait ran out here or in another block.
__device__ __forceinline__ bool gs_wait(const GatedScanParams& p, const unsigned long long* w, GsPair* v) {
  for (unsigned i = 0; gs_empty(*v); ++i) {
    if (i >= kGsMaxPolls || ((i & 255) == 255 && *reinterpret_cast<volatile unsigned*>(p.abort) != kGsEmpty)) {
      if (i >= kGsMaxPolls) flag_status(MATE_DEV_TIMEOUT);
      *reinterpret_cast<volatile unsigned*>(p.abort) = 0u;
      return false;
    }
    if (i > 8) __nanosleep(32);
    *v = gs_look(w);
  }
  return true;
}

template <typename T_>
__device__ __forceinline__ float2 gs_load2(const T_* p);
template <>
__device__ __forceinline__ float2 gs_load2<float>(const float* p) { return *reinterpret_cast<const float2*>(p); }
template <>
__device__ __forceinline__ float2 gs_load2<__nv_bfloat16>(const __nv_bfloat16* p) {
  return unpack_bf16x2(*reinterpret_cast<const uint32_t*>(p));
}
__device__ __forceinline__ void gs_store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void gs_store2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(a, b);
}

// Row `row` behind p; row strides are below 2^31 elements.
template <typename T_>
__device__ __forceinline__ T_* gs_at(T_* p, int row, unsigned ld) {
  return p + static_cast<unsigned long long>(static_cast<unsigned>(row)) * ld;
}

// Short sequences (a token or a few per call): one thread per sample and channel pair, no tiles.
template <typename T_>
__global__ void __launch_bounds__(128) gated_scan_short_kernel(GatedScanParams p) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int half = p.D / 2;
  if (i >= (long long)p.B * half) return;
  const int b = static_cast<int>(i / half), c = 2 * static_cast<int>(i - (long long)b * half);
  float2 x[kGsShort], g[kGsShort];
  int row[kGsShort];
#pragma unroll
  for (int s = 0; s < kGsShort; ++s)
    if (s < p.n) {
      row[s] = gs_row(p, s);
      const long long r = (long long)b * p.n + row[s];
      x[s] = gs_load2(static_cast<const T_*>(p.x) + r * p.ldx + c);
      g[s] = gs_load2(static_cast<const T_*>(p.g) + r * p.ldg + c);
    }
  const float2 zero = make_float2(0.f, 0.f);
  const float2 bias = p.bias != nullptr ? *reinterpret_cast<const float2*>(p.bias + c) : zero;
  float2 h = p.h0 != nullptr ? *reinterpret_cast<const float2*>(p.h0 + (long long)b * p.D + c) : zero;
  if (p.states != nullptr) *reinterpret_cast<float2*>(p.states + (long long)b * p.D + c) = h;
#pragma unroll
  for (int s = 0; s < kGsShort; ++s)
    if (s < p.n) {
      float2 a, na;
      gs_gate(mul_f32x2(add2(g[s], bias), both(kGsLog2e)), &a, &na);
      h = fma2(a, h, mul_f32x2(na, x[s]));
      gs_store2(static_cast<T_*>(p.y) + ((long long)b * p.n + row[s]) * p.ldy + c, h.x, h.y);
    }
  if (p.h_last != nullptr) *reinterpret_cast<float2*>(p.h_last + (long long)b * p.D + c) = h;
}

// Shared memory of a block: a ring of stages with the tiles of NT tensors (x, g and, backward, dy; rows of 64 channels,
// as the TMA gathers lay them down) and what the tile is, then the joins' scratch.
template <typename T_, int NT>
struct GsSmem {
  T_ tile[kGsStages<T_, NT>][NT][kGsRows<T_>][kGsChan];
  alignas(16) int row[kGsStages<T_, NT>][kGsRows<T_>];     // grid row of each step
  int k[kGsStages<T_, NT>], b[kGsStages<T_, NT>], c0[kGsStages<T_, NT>];   // the tile (in working order), -1: no more
  float2 wa[kGsWarps][32], wh[kGsWarps][32];   // the warps' pairs (backward: the adjoint's)
  float2 wf[NT == 3 ? kGsWarps : 1][32];       // backward: the forward pairs' H
  float2 la[kGsWarps][32], lh[kGsWarps][32];   // the pairs that each warp joined from the tiles before
  float2 lg[32];                               // state before the group
  float2 db[NT == 3 ? kGsWarps : 1][32];
  uint64_t full[kGsStages<T_, NT>];
};

struct GsMaps {
  CUtensorMap x, g, dy;   // boxes of one row x 64 channels (fp32: 32), no swizzle
};

// The next ticket of a block, in lane 0 of its loading warp, asked for one tile ahead of its use.  The counter starts at
// ~0, so that the first ticket is 0; a single tile of rows needs no order.
__device__ __forceinline__ unsigned gs_ticket(const GatedScanParams& p, unsigned last) {
  if (p.ticket == nullptr) return last + gridDim.x;
  return (threadIdx.x & 31) == 0 ? atomicAdd(p.ticket, 1u) + 1u : 0u;
}

// Starts the loads of tile t into a stage that no warp reads any more (whole warp); the backward pass (NT = 3) walks the
// tiles from the last rows to the first.
template <typename T_, int NT>
__device__ __forceinline__ void gs_load(const GatedScanParams& p, const GsMaps& maps, GsSmem<T_, NT>& sm, int stage,
                                        unsigned t) {
  constexpr int R = kGsRows<T_>, BC = 128 / sizeof(T_);   // channels per gather
  const int lane = threadIdx.x & 31;
  const unsigned total = static_cast<unsigned>(p.tiles) * p.B * p.cblocks, per = static_cast<unsigned>(p.B) * p.cblocks;
  t = __shfl_sync(0xffffffffu, t, 0);
  const bool more = t < total;
  const unsigned k = t / per, r = t - k * per;
  const int b = r / p.cblocks, c0 = (r % p.cblocks) * kGsChan;
  const int s0 = (NT == 3 ? p.tiles - 1 - static_cast<int>(k) : static_cast<int>(k)) * R;
  int row[R / 32];
  if (more) {
#pragma unroll
    for (int j = 0; j < R / 32; ++j) {
      const int s = s0 + lane * (R / 32) + j;
      row[j] = s < p.n ? gs_row(p, s) : -1;
      sm.row[stage][lane * (R / 32) + j] = row[j];
    }
  }
  if (lane == 0) {
    sm.k[stage] = more ? static_cast<int>(k) : -1;
    sm.b[stage] = b;
    sm.c0[stage] = c0;
  }
  __syncwarp();
  if (lane == 0) {
    if (more) mbar_arrive_expect_tx(&sm.full[stage], NT * R * kGsChan * sizeof(T_));
    else mbar_arrive(&sm.full[stage]);
  }
  if (!more) return;
  __syncwarp();
  // four rows per gather; a row behind the last reads zeros (a row index behind the tensor)
  const int none = p.B * p.n, base = b * p.n;
  if constexpr (R / 32 == 4) {
    const int r0 = row[0] < 0 ? none : base + row[0], r1 = row[1] < 0 ? none : base + row[1];
    const int r2 = row[2] < 0 ? none : base + row[2], r3 = row[3] < 0 ? none : base + row[3];
    tma_gather4(&maps.x, &sm.full[stage], &sm.tile[stage][0][lane * 4][0], c0, r0, r1, r2, r3);
    tma_gather4(&maps.g, &sm.full[stage], &sm.tile[stage][1][lane * 4][0], c0, r0, r1, r2, r3);
    if constexpr (NT == 3)
      tma_gather4(&maps.dy, &sm.full[stage], &sm.tile[stage][2][lane * 4][0], c0, r0, r1, r2, r3);
  } else {
    // 64 rows of fp32: lane l gathers the rows of lanes 2q, 2q + 1 (q = l / 2), half of the channels (a gather's rows
    // lie 128 bytes apart, so a tile holds its two halves of 32 channels one behind the other)
    const int q = lane >> 1, hf = lane & 1;
    int rr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = __shfl_sync(0xffffffffu, row[j & 1], 2 * q + (j >> 1));
      rr[j] = v < 0 ? none : base + v;
    }
    const int off = hf * R * BC + q * 4 * BC;
    tma_gather4(&maps.x, &sm.full[stage], &sm.tile[stage][0][0][0] + off, c0 + hf * BC, rr[0], rr[1], rr[2], rr[3]);
    tma_gather4(&maps.g, &sm.full[stage], &sm.tile[stage][1][0][0] + off, c0 + hf * BC, rr[0], rr[1], rr[2], rr[3]);
    if constexpr (NT == 3)
      tma_gather4(&maps.dy, &sm.full[stage], &sm.tile[stage][2][0][0] + off, c0 + hf * BC, rr[0], rr[1], rr[2], rr[3]);
  }
}

// A thread's two channels of row r of a stage's tile.
template <typename T_, int NT>
__device__ __forceinline__ float2 gs_elem(const GsSmem<T_, NT>& sm, int stage, int tensor, int r, int lane) {
  constexpr int BC = 128 / sizeof(T_);
  const T_* base = &sm.tile[stage][tensor][0][0];
  return gs_load2(base + ((2 * lane) / BC) * (kGsRows<T_> * BC) + r * BC + (2 * lane) % BC);
}

// Joins the tiles before tile k of its group: warp w takes tiles 4w .. 4w + 3, the last warp the group's state too.
// Returns false if a wait ran out.
template <typename T_, int NT>
__device__ __forceinline__ bool gs_before(const GatedScanParams& p, GsSmem<T_, NT>& sm, int k, long long at, bool live,
                                          float2 start) {
  constexpr int per = kGsGroup / kGsWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m = k % kGsGroup, j0 = warp * per;
  const long long step = (long long)p.B * p.D;
  float2 A = both(1.f), H = both(0.f);
  bool ok = true;
  if (live) {
    const unsigned long long* w = p.pair + (k - m + j0) * step + at;
    GsPair v[per];
#pragma unroll
    for (int j = 0; j < per; ++j)
      if (j0 + j < m) v[j] = gs_look(w + j * step);
    if (warp == kGsWarps - 1) {
      if (k >= kGsGroup) {
        const unsigned long long* wg = p.group + (k / kGsGroup) * step + at;
        GsPair g = gs_look(wg);
        ok = gs_wait(p, wg, &g);
        start = make_float2(f2_from(g.x).y, f2_from(g.y).y);
      }
      sm.lg[lane] = start;
    }
#pragma unroll
    for (int j = 0; j < per; ++j)
      if (j0 + j < m && ok) {
        ok = gs_wait(p, w + j * step, &v[j]);
        const float2 u = f2_from(v[j].x), q = f2_from(v[j].y);
        H = fma2(make_float2(u.x, q.x), H, make_float2(u.y, q.y));
        A = mul_f32x2(A, make_float2(u.x, q.x));
      }
  }
  if (j0 < m) {
    sm.la[warp][lane] = A;
    sm.lh[warp][lane] = H;
  }
  return ok;
}

// The state before the tile, from what gs_before left.
template <typename T_, int NT>
__device__ __forceinline__ float2 gs_carry(const GsSmem<T_, NT>& sm, int k, int lane) {
  constexpr int per = kGsGroup / kGsWarps;
  float2 h = sm.lg[lane];
  const int used = (k % kGsGroup + per - 1) / per;
#pragma unroll
  for (int w = 0; w < kGsWarps; ++w)
    if (w < used) h = fma2(sm.la[w][lane], h, sm.lh[w][lane]);
  return h;
}

template <typename T_, int NT>
__device__ __forceinline__ void gs_init(GsSmem<T_, NT>& sm, const GsMaps& maps) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGsStages<T_, NT>; ++s) {
      mbar_init(&sm.full[s], 1);
    }
    mbar_fence_init();
    prefetch_tensormap(&maps.x);
    prefetch_tensormap(&maps.g);
    if (NT == 3) prefetch_tensormap(&maps.dy);
  }
  __syncthreads();
}

template <typename T_>
__global__ void __launch_bounds__(kGsThreads, 2)
    gated_scan_kernel(const __grid_constant__ GsMaps maps, const GatedScanParams p) {
  extern __shared__ __align__(128) uint8_t gs_raw[];
  GsSmem<T_, 2>& sm = *reinterpret_cast<GsSmem<T_, 2>*>(gs_raw);
  constexpr int RUN = kGsRun<T_>, S = kGsStages<T_, 2>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  gs_init(sm, maps);
  unsigned ticket = 0;
  if (warp == kGsLoadWarp) {
    ticket = gs_ticket(p, blockIdx.x - gridDim.x);
    for (int s = 0; s < S - 1; ++s) {
      gs_load(p, maps, sm, s, ticket);
      ticket = gs_ticket(p, ticket);
    }
  }
  const float2 zero = both(0.f), one = both(1.f);
  const long long step = (long long)p.B * p.D;
  bool dead = false;   // a wait ran out: the remaining tiles are only taken off the ring
  for (int it = 0;; ++it) {
    const int stage = it % S;
    if (!mbar_wait(&sm.full[stage], (it / S) & 1)) break;
    const int k = sm.k[stage];
    if (k < 0) break;
    const int b = sm.b[stage], c = sm.c0[stage] + 2 * lane;
    const bool live = c < p.D && !dead;
    const long long at = (long long)b * p.D + c;
    const float2 bias = mul_f32x2(
        live && p.bias != nullptr ? *reinterpret_cast<const float2*>(p.bias + c) : zero, both(kGsLog2e));
    const int rows = p.n - (k * kGsRows<T_> + warp * RUN);   // of this warp, RUN at most; the rest keep the state
    float2 a[RUN], v[RUN];
    float2 A = one, H = zero;
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      float2 na;
      gs_gate(fma2(gs_elem(sm, stage, 1, warp * RUN + r, lane), both(kGsLog2e), bias), &a[r], &na);
      v[r] = mul_f32x2(na, gs_elem(sm, stage, 0, warp * RUN + r, lane));
    }
    if (rows < RUN) {
#pragma unroll
      for (int r = 0; r < RUN; ++r)
        if (r >= rows) {
          a[r] = one;
          v[r] = zero;
        }
    }
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      H = fma2(a[r], H, v[r]);
      A = mul_f32x2(A, a[r]);
    }
    sm.wa[warp][lane] = A;
    sm.wh[warp][lane] = H;
    __syncthreads();
    if (warp == kGsLoadWarp) {   // all warps are done with the tile before this one: its stage takes the next
      gs_load(p, maps, sm, (it + S - 1) % S, ticket);
      ticket = gs_ticket(p, ticket);
    }
    // pairs of the warps before this one; the first warp forms the whole tile's
    float2 Ab = one, Hb = zero;
#pragma unroll
    for (int w = 0; w < kGsWarps; ++w)
      if (w < warp || warp == 0) {
        const float2 aw = sm.wa[w][lane];
        Hb = fma2(aw, Hb, sm.wh[w][lane]);
        Ab = mul_f32x2(Ab, aw);
      }
    if (warp == 0 && live && k + 1 < p.tiles) gs_publish(p.pair + k * step + at, Ab, Hb);
    const float2 h0 = live && p.h0 != nullptr ? *reinterpret_cast<const float2*>(p.h0 + at) : zero;
    dead = __syncthreads_or(!gs_before(p, sm, k, at, live, h0) || dead);
    if (!dead && live) {
      float2 h = gs_carry(sm, k, lane);
      if (warp == 0) {
        if (p.states != nullptr) *reinterpret_cast<float2*>(p.states + ((long long)b * p.tiles + k) * p.D + c) = h;
        const float2 out = fma2(Ab, h, Hb);
        if (k + 1 == p.tiles) {
          if (p.h_last != nullptr) *reinterpret_cast<float2*>(p.h_last + at) = out;
        } else if ((k + 1) % kGsGroup == 0) {
          gs_publish(p.group + (k + 1) / kGsGroup * step + at, zero, out);
        }
      } else {
        h = fma2(Ab, h, Hb);
      }
      T_* y = static_cast<T_*>(p.y) + (long long)b * p.n * p.ldy + c;
      if (rows >= RUN) {
#pragma unroll
        for (int r = 0; r < RUN; r += 4) {
          const int4 row = *reinterpret_cast<const int4*>(&sm.row[stage][warp * RUN + r]);
          h = fma2(a[r], h, v[r]);
          gs_store2(gs_at(y, row.x, p.ldy), h.x, h.y);
          h = fma2(a[r + 1], h, v[r + 1]);
          gs_store2(gs_at(y, row.y, p.ldy), h.x, h.y);
          h = fma2(a[r + 2], h, v[r + 2]);
          gs_store2(gs_at(y, row.z, p.ldy), h.x, h.y);
          h = fma2(a[r + 3], h, v[r + 3]);
          gs_store2(gs_at(y, row.w, p.ldy), h.x, h.y);
        }
      } else {
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
          h = fma2(a[r], h, v[r]);
          if (r < rows) gs_store2(gs_at(y, sm.row[stage][warp * RUN + r], p.ldy), h.x, h.y);
        }
      }
    }
  }
}

// The backward pass: tiles from the last rows to the first; the state before each row is formed again from the saved
// state before the tile, the adjoint state joins like the forward's (m -> A m + M from the row behind to the row before).
template <typename T_>
__global__ void __launch_bounds__(kGsThreads, 2)
    gated_scan_bwd_kernel(const __grid_constant__ GsMaps maps, const GatedScanParams p) {
  extern __shared__ __align__(128) uint8_t gs_raw[];
  GsSmem<T_, 3>& sm = *reinterpret_cast<GsSmem<T_, 3>*>(gs_raw);
  constexpr int RUN = kGsRun<T_>, S = kGsStages<T_, 3>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  gs_init(sm, maps);
  unsigned ticket = 0;
  if (warp == kGsLoadWarp) {
    ticket = gs_ticket(p, blockIdx.x - gridDim.x);
    for (int s = 0; s < S - 1; ++s) {
      gs_load(p, maps, sm, s, ticket);
      ticket = gs_ticket(p, ticket);
    }
  }
  const float2 zero = both(0.f), one = both(1.f), neg = both(-1.f);
  const long long step = (long long)p.B * p.D;
  bool dead = false;
  for (int it = 0;; ++it) {
    const int stage = it % S;
    if (!mbar_wait(&sm.full[stage], (it / S) & 1)) break;
    const int k = sm.k[stage];
    if (k < 0) break;
    const int kr = p.tiles - 1 - k;   // the tile of rows
    const int b = sm.b[stage], c = sm.c0[stage] + 2 * lane;
    const bool live = c < p.D && !dead;
    const long long at = (long long)b * p.D + c;
    const float2 bias = mul_f32x2(
        live && p.bias != nullptr ? *reinterpret_cast<const float2*>(p.bias + c) : zero, both(kGsLog2e));
    const float2 h_in = live ? *reinterpret_cast<const float2*>(p.states + ((long long)b * p.tiles + kr) * p.D + c) : zero;
    const int rows = p.n - (kr * kGsRows<T_> + warp * RUN);
    float2 a[RUN], na[RUN];
    float2 A = one, H = zero, Mm = zero;
#pragma unroll
    for (int r = 0; r < RUN; ++r)
      gs_gate(fma2(gs_elem(sm, stage, 1, warp * RUN + r, lane), both(kGsLog2e), bias), &a[r], &na[r]);
    if (rows < RUN) {
#pragma unroll
      for (int r = 0; r < RUN; ++r)
        if (r >= rows) {
          a[r] = one;
          na[r] = zero;
        }
    }
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      H = fma2(a[r], H, mul_f32x2(na[r], gs_elem(sm, stage, 0, warp * RUN + r, lane)));
      A = mul_f32x2(A, a[r]);
    }
#pragma unroll
    for (int r = RUN - 1; r >= 0; --r) Mm = mul_f32x2(a[r], add2(gs_elem(sm, stage, 2, warp * RUN + r, lane), Mm));
    sm.wa[warp][lane] = A;
    sm.wf[warp][lane] = H;
    sm.wh[warp][lane] = Mm;
    __syncthreads();
    if (warp == kGsLoadWarp) {
      gs_load(p, maps, sm, (it + S - 1) % S, ticket);
      ticket = gs_ticket(p, ticket);
    }
    // adjoint pairs of the warps behind this one (the last warp: of the whole tile); the state before this warp's rows
    float2 Ab = one, Mb = zero, h = h_in;
#pragma unroll
    for (int q = kGsWarps - 1; q >= 0; --q)
      if (q > warp || warp == kGsWarps - 1) {
        const float2 aw = sm.wa[q][lane];
        Mb = fma2(aw, Mb, sm.wh[q][lane]);
        Ab = mul_f32x2(Ab, aw);
      }
    if (warp == kGsWarps - 1 && live && k + 1 < p.tiles) gs_publish(p.pair + k * step + at, Ab, Mb);
#pragma unroll
    for (int q = 0; q < kGsWarps - 1; ++q)
      if (q < warp) h = fma2(sm.wa[q][lane], h, sm.wf[q][lane]);
    const float2 m0 = live && p.dh_last != nullptr ? *reinterpret_cast<const float2*>(p.dh_last + at) : zero;
    dead = __syncthreads_or(!gs_before(p, sm, k, at, live, m0) || dead);
    float2 db = zero;
    if (!dead && live) {
      float2 m = gs_carry(sm, k, lane);
      if (warp == kGsWarps - 1) {
        const float2 out = fma2(Ab, m, Mb);
        if (k + 1 == p.tiles) {
          if (p.dh0 != nullptr) *reinterpret_cast<float2*>(p.dh0 + at) = out;
        } else if ((k + 1) % kGsGroup == 0) {
          gs_publish(p.group + (k + 1) / kGsGroup * step + at, zero, out);
        }
      } else {
        m = fma2(Ab, m, Mb);
      }
      // the state before each row, less x
      float2 w[RUN];
#pragma unroll
      for (int r = 0; r < RUN; ++r) {
        const float2 x = gs_elem(sm, stage, 0, warp * RUN + r, lane);
        w[r] = fma2(x, neg, h);
        h = fma2(a[r], h, mul_f32x2(na[r], x));
      }
      T_* dx = static_cast<T_*>(p.dx) + (long long)b * p.n * p.lddx + c;
      T_* dg = static_cast<T_*>(p.dg) + (long long)b * p.n * p.lddg + c;
#pragma unroll
      for (int r = RUN - 1; r >= 0; --r) {
        const float2 l = add2(gs_elem(sm, stage, 2, warp * RUN + r, lane), m);
        const float2 o = mul_f32x2(na[r], l);
        m = mul_f32x2(a[r], l);
        const float2 d = mul_f32x2(mul_f32x2(o, w[r]), a[r]);
        if (r < rows) {
          const int row = sm.row[stage][warp * RUN + r];
          gs_store2(gs_at(dx, row, p.lddx), o.x, o.y);
          gs_store2(gs_at(dg, row, p.lddg), d.x, d.y);
          db = add2(db, d);
        }
      }
    }
    if (p.dbias_part != nullptr) {
      sm.db[warp][lane] = db;
      __syncthreads();
      if (warp == 0 && live && !dead) {
        float2 v = zero;
#pragma unroll
        for (int q = 0; q < kGsWarps; ++q) v = add2(v, sm.db[q][lane]);
        *reinterpret_cast<float2*>(p.dbias_part + ((long long)b * p.tiles + kr) * p.D + c) = v;
      }
    }
  }
}

}  // namespace mate
