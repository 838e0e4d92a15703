// Gated linear recurrence over the grid's tokens in one of the four scan orders, and its backward pass (an
// elementwise-state companion of the selective scan; the pages describe only the latter).  Per sample and channel:
//   a_t = sigmoid(g_t + bias),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  y_t = h_t            (h_0 given or zero)
// Backward, with the adjoint state l_t = dy_t + m_{t+1}, m_t = a_t l_t (behind the last row: m = gradient of h_last):
//   dx_t = (1 - a_t) l_t,  dg_t = l_t (h_{t-1} - x_t) a_t (1 - a_t),  dbias = sum of dg,  dh0 = m_1.
// States, gates and sums are fp32; y, dx and dg are rounded once on the way out.
//
// One pass over the data.  A tile is kGsRows steps x 64 channels; a run of rows maps the state before it to the state
// behind it by h -> A h + H, and such pairs (A, H) join in order.  Persistent blocks take tiles by ticket (all
// channels and samples of the first rows, then the next rows), prefetch the next tile's rows into shared memory,
// form the tile's pair, publish it, and find the state before the tile from the pairs of the tiles before it in its
// group of kGsGroup tiles and the state before that group, which the last tile of the group before publishes.  The
// joins are the same ones in the same order on every run, whoever publishes first, so the result is reproducible.
// A ticket only waits for smaller tickets, and a block works its tickets off in order, so the smallest unfinished
// tile can always finish: nothing depends on how many blocks run at a time.
#pragma once
#include "common.cuh"
#include "mamba_extras.cuh"   // to_f32, from_f32

namespace mate {

constexpr int kGsRows = 64;            // steps per tile; the forward's `states` hold the state before each tile
constexpr int kGsChan = 64;            // channels per tile: 32 lanes x 2
constexpr int kGsWarps = 8;
constexpr int kGsThreads = kGsWarps * 32;
constexpr int kGsRun = kGsRows / kGsWarps;   // consecutive steps per thread
constexpr int kGsGroup = 32;           // tiles per group: at most 31 pairs to join behind the group's state
constexpr int kGsShort = 8;            // longest sequence of the short kernel

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

// The smaller of sigmoid(z) and sigmoid(-z), with the sign bit set if it is sigmoid(z): one register holds both, each
// to full precision (the other is one minus it, at least 1/2).
__device__ __forceinline__ float gs_gate(float z) {
  const float e = ex2_approx(-1.4426950408889634f * fabsf(z));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  const float s = e * r;
  return z < 0.f ? -s : s;
}
__device__ __forceinline__ void gs_split(float s, float* a, float* na) {
  const float t = fabsf(s), u = 1.f - t;
  const bool neg = __float_as_int(s) < 0;
  *a = neg ? t : u;
  *na = neg ? u : t;
}

__device__ __forceinline__ unsigned long long gs_pack(float lo, float hi) {
  return (static_cast<unsigned long long>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
}
// Data and validity travel in one 64-bit word, so publishing needs no fence and reading no second look.
__device__ __forceinline__ void gs_publish(unsigned long long* w, unsigned long long v) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(w), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long gs_look(const unsigned long long* w) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(w) : "memory");
  return v;
}
constexpr unsigned kGsMaxPolls = 1u << 20;   // about a second

// Waits until both words are published; false if the wait ran out here or in another block.
__device__ __forceinline__ bool gs_wait(const GatedScanParams& p, const unsigned long long* w, unsigned long long v[2]) {
  for (unsigned i = 0; static_cast<unsigned>(v[0]) == kGsEmpty || static_cast<unsigned>(v[1]) == kGsEmpty; ++i) {
    if (i >= kGsMaxPolls || ((i & 255) == 255 && *reinterpret_cast<volatile unsigned*>(p.abort) != kGsEmpty)) {
      if (i >= kGsMaxPolls) flag_status(MATE_DEV_TIMEOUT);
      *reinterpret_cast<volatile unsigned*>(p.abort) = 0u;
      return false;
    }
    if (i > 8) __nanosleep(32);
    v[0] = gs_look(w);
    v[1] = gs_look(w + 1);
  }
  return true;
}
__device__ __forceinline__ float gs_lo(unsigned long long v) { return __uint_as_float(static_cast<unsigned>(v)); }
__device__ __forceinline__ float gs_hi(unsigned long long v) { return __uint_as_float(static_cast<unsigned>(v >> 32)); }
// A pair's low word may not look empty: a NaN gets the payload that arithmetic gives it.
__device__ __forceinline__ float gs_clean(float a) { return a != a ? __uint_as_float(0x7fffffffu) : a; }

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
      float a, na;
      gs_split(gs_gate(g[s].x + bias.x), &a, &na);
      h.x = fmaf(a, h.x, na * x[s].x);
      gs_split(gs_gate(g[s].y + bias.y), &a, &na);
      h.y = fmaf(a, h.y, na * x[s].y);
      gs_store2(static_cast<T_*>(p.y) + ((long long)b * p.n + row[s]) * p.ldy + c, h.x, h.y);
    }
  if (p.h_last != nullptr) *reinterpret_cast<float2*>(p.h_last + (long long)b * p.D + c) = h;
}

// Shared memory of a block: two stages of NT tensors' tiles, then the joins' scratch.
template <typename T_, int NT>
struct GsSmem {
  T_ tile[2][NT][kGsRows][kGsChan];
  int row[2][kGsRows];                    // grid row of each step, -1 behind the last
  float2 wa[kGsWarps][32], wh[kGsWarps][32];   // the warps' pairs (and forward pairs, backward)
  float2 wf[NT == 3 ? kGsWarps : 1][32];
  float2 la[kGsWarps][32], lh[kGsWarps][32];   // the pairs that each warp joined from the tiles before
  float2 lg[32];                          // state before the group
  float2 db[NT == 3 ? kGsWarps : 1][32];
  unsigned next;
};

struct GsTile {
  int k, b, c0;   // k-th tile of rows in the order they are worked off
};
__device__ __forceinline__ GsTile gs_tile(const GatedScanParams& p, unsigned t) {
  const unsigned per = static_cast<unsigned>(p.B) * p.cblocks;
  const unsigned k = t / per, r = t - k * per;
  return {static_cast<int>(k), static_cast<int>(r / p.cblocks), static_cast<int>(r % p.cblocks) * kGsChan};
}

// Copies the rows [k * kGsRows, ..) of the tensors into a stage.
template <typename T_, int NT>
__device__ __forceinline__ void gs_fetch(const GatedScanParams& p, GsSmem<T_, NT>& sm, int stage, int k, int b, int c0) {
  constexpr int V = 16 / sizeof(T_), PER = kGsChan / V;
#pragma unroll
  for (int i = threadIdx.x; i < kGsRows * PER; i += kGsThreads) {
    const int r = i / PER, v = i % PER, s = k * kGsRows + r;
    const int row = s < p.n ? gs_row(p, s) : -1;
    if (v == 0) sm.row[stage][r] = row;
    const bool ok = row >= 0 && c0 + v * V < p.D;
    const long long at = (long long)b * p.n + row;
    cp_async16_zfill(&sm.tile[stage][0][r][v * V], ok ? static_cast<const T_*>(p.x) + at * p.ldx + c0 + v * V : p.x, ok);
    cp_async16_zfill(&sm.tile[stage][1][r][v * V], ok ? static_cast<const T_*>(p.g) + at * p.ldg + c0 + v * V : p.g, ok);
    if constexpr (NT == 3)
      cp_async16_zfill(&sm.tile[stage][2][r][v * V], ok ? static_cast<const T_*>(p.dy) + at * p.lddy + c0 + v * V : p.dy,
                       ok);
  }
  cp_async_commit();
}

// Joins the tiles before tile k of its group: warp w takes tiles 4w .. 4w + 3, the last warp the group's state too.
// Returns false if a wait ran out.
template <typename T_, int NT>
__device__ __forceinline__ bool gs_before(const GatedScanParams& p, GsSmem<T_, NT>& sm, int k, int b, int c, bool live,
                                          float2 start) {
  constexpr int per = kGsGroup / kGsWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = k / kGsGroup * kGsGroup, m = k - k0;
  const long long step = (long long)p.B * p.D, at = (long long)b * p.D + c;
  float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f);
  bool ok = true;
  if (live) {
    unsigned long long v[per][2];
#pragma unroll
    for (int j = 0; j < per; ++j)
      if (warp * per + j < m) {
        const unsigned long long* w = p.pair + (k0 + warp * per + j) * step + at;
        v[j][0] = gs_look(w);
        v[j][1] = gs_look(w + 1);
      }
    if (warp == kGsWarps - 1) {
      float2 h = start;
      if (k0 > 0) {
        const unsigned long long* w = p.group + (k / kGsGroup) * step + at;
        unsigned long long g[2] = {gs_look(w), gs_look(w + 1)};
        ok = gs_wait(p, w, g);
        h = make_float2(gs_hi(g[0]), gs_hi(g[1]));
      }
      sm.lg[lane] = h;
    }
#pragma unroll
    for (int j = 0; j < per; ++j)
      if (warp * per + j < m && ok) {
        ok = gs_wait(p, p.pair + (k0 + warp * per + j) * step + at, v[j]);
        H.x = fmaf(gs_lo(v[j][0]), H.x, gs_hi(v[j][0]));
        H.y = fmaf(gs_lo(v[j][1]), H.y, gs_hi(v[j][1]));
        A.x *= gs_lo(v[j][0]);
        A.y *= gs_lo(v[j][1]);
      }
  }
  sm.la[warp][lane] = A;
  sm.lh[warp][lane] = H;
  return ok;
}

// The state before the tile, from what gs_before left.
template <typename T_, int NT>
__device__ __forceinline__ float2 gs_carry(const GsSmem<T_, NT>& sm, int k, int lane) {
  float2 h = sm.lg[lane];
  const int used = (k % kGsGroup + kGsGroup / kGsWarps - 1) / (kGsGroup / kGsWarps);
  for (int w = 0; w < used; ++w) {
    h.x = fmaf(sm.la[w][lane].x, h.x, sm.lh[w][lane].x);
    h.y = fmaf(sm.la[w][lane].y, h.y, sm.lh[w][lane].y);
  }
  return h;
}

template <typename T_>
__global__ void __launch_bounds__(kGsThreads, sizeof(T_) == 2 ? 4 : 3) gated_scan_kernel(const GatedScanParams p) {
  extern __shared__ __align__(128) uint8_t gs_raw[];
  GsSmem<T_, 2>& sm = *reinterpret_cast<GsSmem<T_, 2>*>(gs_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned total = static_cast<unsigned>(p.tiles) * p.B * p.cblocks;
  const float2 zero = make_float2(0.f, 0.f);
  // tickets: the counter starts at ~0, so that the first one is 0; a single tile of rows needs no order
  if (threadIdx.x == 0) sm.next = p.ticket != nullptr ? atomicAdd(p.ticket, 1u) + 1u : blockIdx.x;
  __syncthreads();
  unsigned cur = sm.next;
  int stage = 0;
  GsTile t = gs_tile(p, cur);
  if (cur < total) gs_fetch(p, sm, 0, t.k, t.b, t.c0);
  __syncthreads();
  while (cur < total) {
    if (threadIdx.x == 0) sm.next = p.ticket != nullptr ? atomicAdd(p.ticket, 1u) + 1u : cur + gridDim.x;
    const int c = t.c0 + 2 * lane;
    const bool live = c < p.D;
    const float2 bias = live && p.bias != nullptr ? *reinterpret_cast<const float2*>(p.bias + c) : zero;
    cp_async_wait<0>();
    __syncthreads();
    const unsigned nxt = sm.next;
    const GsTile u = gs_tile(p, nxt);
    if (nxt < total) gs_fetch(p, sm, stage ^ 1, u.k, u.b, u.c0);
    float2 a[kGsRun], v[kGsRun];
    float2 A = make_float2(1.f, 1.f), H = zero;
#pragma unroll
    for (int r = 0; r < kGsRun; ++r) {
      const float2 x = gs_load2(&sm.tile[stage][0][warp * kGsRun + r][2 * lane]);
      const float2 g = gs_load2(&sm.tile[stage][1][warp * kGsRun + r][2 * lane]);
      float2 na;
      gs_split(gs_gate(g.x + bias.x), &a[r].x, &na.x);
      gs_split(gs_gate(g.y + bias.y), &a[r].y, &na.y);
      v[r] = make_float2(na.x * x.x, na.y * x.y);
      if (sm.row[stage][warp * kGsRun + r] < 0) {   // behind the last row: the state stays
        a[r] = make_float2(1.f, 1.f);
        v[r] = zero;
      }
      H = make_float2(fmaf(a[r].x, H.x, v[r].x), fmaf(a[r].y, H.y, v[r].y));
      A = make_float2(A.x * a[r].x, A.y * a[r].y);
    }
    sm.wa[warp][lane] = A;
    sm.wh[warp][lane] = H;
    __syncthreads();
    // pairs of the warps before this one, and of the whole tile
    float2 Ab = make_float2(1.f, 1.f), Hb = zero, At = Ab, Ht = zero;
#pragma unroll
    for (int w = 0; w < kGsWarps; ++w) {
      if (w == warp) {
        Ab = At;
        Hb = Ht;
      }
      const float2 aw = sm.wa[w][lane], hw = sm.wh[w][lane];
      Ht = make_float2(fmaf(aw.x, Ht.x, hw.x), fmaf(aw.y, Ht.y, hw.y));
      At = make_float2(At.x * aw.x, At.y * aw.y);
    }
    const long long step = (long long)p.B * p.D, at = (long long)t.b * p.D + c;
    if (warp == 0 && live && t.k + 1 < p.tiles) {
      gs_publish(p.pair + t.k * step + at, gs_pack(gs_clean(At.x), Ht.x));
      gs_publish(p.pair + t.k * step + at + 1, gs_pack(gs_clean(At.y), Ht.y));
    }
    const float2 h0 = live && p.h0 != nullptr ? *reinterpret_cast<const float2*>(p.h0 + at) : zero;
    if (__syncthreads_or(!gs_before(p, sm, t.k, t.b, c, live, h0))) break;
    const float2 h_in = gs_carry(sm, t.k, lane);
    if (warp == 0 && live) {
      if (p.states != nullptr) *reinterpret_cast<float2*>(p.states + ((long long)t.b * p.tiles + t.k) * p.D + c) = h_in;
      const float2 out = make_float2(fmaf(At.x, h_in.x, Ht.x), fmaf(At.y, h_in.y, Ht.y));
      if (t.k + 1 == p.tiles) {
        if (p.h_last != nullptr) *reinterpret_cast<float2*>(p.h_last + at) = out;
      } else if ((t.k + 1) % kGsGroup == 0) {
        gs_publish(p.group + (t.k + 1) / kGsGroup * step + at, gs_pack(0.f, out.x));
        gs_publish(p.group + (t.k + 1) / kGsGroup * step + at + 1, gs_pack(0.f, out.y));
      }
    }
    if (live) {
      float2 h = make_float2(fmaf(Ab.x, h_in.x, Hb.x), fmaf(Ab.y, h_in.y, Hb.y));
#pragma unroll
      for (int r = 0; r < kGsRun; ++r) {
        h = make_float2(fmaf(a[r].x, h.x, v[r].x), fmaf(a[r].y, h.y, v[r].y));
        const int row = sm.row[stage][warp * kGsRun + r];
        if (row >= 0) gs_store2(static_cast<T_*>(p.y) + ((long long)t.b * p.n + row) * p.ldy + c, h.x, h.y);
      }
    }
    cur = nxt;
    t = u;
    stage ^= 1;
  }
  cp_async_wait<0>();
}

// The backward pass: tiles from the last rows to the first; the state before each row is formed again from the saved
// state before the tile, the adjoint state joins like the forward's (m -> A m + M from the row behind to the row before).
template <typename T_>
__global__ void __launch_bounds__(kGsThreads, sizeof(T_) == 2 ? 3 : 2) gated_scan_bwd_kernel(const GatedScanParams p) {
  extern __shared__ __align__(128) uint8_t gs_raw[];
  GsSmem<T_, 3>& sm = *reinterpret_cast<GsSmem<T_, 3>*>(gs_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned total = static_cast<unsigned>(p.tiles) * p.B * p.cblocks;
  const float2 zero = make_float2(0.f, 0.f);
  if (threadIdx.x == 0) sm.next = p.ticket != nullptr ? atomicAdd(p.ticket, 1u) + 1u : blockIdx.x;
  __syncthreads();
  unsigned cur = sm.next;
  int stage = 0;
  GsTile t = gs_tile(p, cur);
  if (cur < total) gs_fetch(p, sm, 0, p.tiles - 1 - t.k, t.b, t.c0);
  __syncthreads();
  while (cur < total) {
    if (threadIdx.x == 0) sm.next = p.ticket != nullptr ? atomicAdd(p.ticket, 1u) + 1u : cur + gridDim.x;
    const int kr = p.tiles - 1 - t.k;   // the tile of rows
    const int c = t.c0 + 2 * lane;
    const bool live = c < p.D;
    const long long step = (long long)p.B * p.D, at = (long long)t.b * p.D + c;
    const float2 bias = live && p.bias != nullptr ? *reinterpret_cast<const float2*>(p.bias + c) : zero;
    const float2 h_in =
        live ? *reinterpret_cast<const float2*>(p.states + ((long long)t.b * p.tiles + kr) * p.D + c) : zero;
    cp_async_wait<0>();
    __syncthreads();
    const unsigned nxt = sm.next;
    const GsTile u = gs_tile(p, nxt);
    if (nxt < total) gs_fetch(p, sm, stage ^ 1, p.tiles - 1 - u.k, u.b, u.c0);
    float2 s[kGsRun], w[kGsRun];   // gate; first (1 - a) x, then the state before the row minus x
    float2 A = make_float2(1.f, 1.f), H = zero, Mm = zero;
#pragma unroll
    for (int r = 0; r < kGsRun; ++r) {
      const float2 x = gs_load2(&sm.tile[stage][0][warp * kGsRun + r][2 * lane]);
      const float2 g = gs_load2(&sm.tile[stage][1][warp * kGsRun + r][2 * lane]);
      s[r] = make_float2(gs_gate(g.x + bias.x), gs_gate(g.y + bias.y));
      if (sm.row[stage][warp * kGsRun + r] < 0) s[r] = zero;   // behind the last row: a = 1
      float2 a, na;
      gs_split(s[r].x, &a.x, &na.x);
      gs_split(s[r].y, &a.y, &na.y);
      H = make_float2(fmaf(a.x, H.x, na.x * x.x), fmaf(a.y, H.y, na.y * x.y));
      A = make_float2(A.x * a.x, A.y * a.y);
    }
#pragma unroll
    for (int r = kGsRun - 1; r >= 0; --r) {
      const float2 dy = gs_load2(&sm.tile[stage][2][warp * kGsRun + r][2 * lane]);
      float2 a, na;
      gs_split(s[r].x, &a.x, &na.x);
      gs_split(s[r].y, &a.y, &na.y);
      Mm = make_float2(a.x * (dy.x + Mm.x), a.y * (dy.y + Mm.y));
    }
    sm.wa[warp][lane] = A;
    sm.wf[warp][lane] = H;
    sm.wh[warp][lane] = Mm;
    __syncthreads();
    // adjoint pairs of the warps behind this one and of the whole tile; the state before this warp's rows
    float2 Ab = make_float2(1.f, 1.f), Mb = zero, At = Ab, Mt = zero, h = h_in;
#pragma unroll
    for (int q = kGsWarps - 1; q >= 0; --q) {
      if (q == warp) {
        Ab = At;
        Mb = Mt;
      }
      const float2 aw = sm.wa[q][lane], mw = sm.wh[q][lane];
      Mt = make_float2(fmaf(aw.x, Mt.x, mw.x), fmaf(aw.y, Mt.y, mw.y));
      At = make_float2(At.x * aw.x, At.y * aw.y);
    }
    if (warp == 0 && live && t.k + 1 < p.tiles) {
      gs_publish(p.pair + t.k * step + at, gs_pack(gs_clean(At.x), Mt.x));
      gs_publish(p.pair + t.k * step + at + 1, gs_pack(gs_clean(At.y), Mt.y));
    }
#pragma unroll
    for (int q = 0; q < kGsWarps - 1; ++q)
      if (q < warp) {
        const float2 aw = sm.wa[q][lane], hw = sm.wf[q][lane];
        h = make_float2(fmaf(aw.x, h.x, hw.x), fmaf(aw.y, h.y, hw.y));
      }
#pragma unroll
    for (int r = 0; r < kGsRun; ++r) {
      const float2 x = gs_load2(&sm.tile[stage][0][warp * kGsRun + r][2 * lane]);
      w[r] = make_float2(h.x - x.x, h.y - x.y);
      float2 a, na;
      gs_split(s[r].x, &a.x, &na.x);
      gs_split(s[r].y, &a.y, &na.y);
      h = make_float2(fmaf(a.x, h.x, na.x * x.x), fmaf(a.y, h.y, na.y * x.y));
    }
    const float2 m0 = live && p.dh_last != nullptr ? *reinterpret_cast<const float2*>(p.dh_last + at) : zero;
    if (__syncthreads_or(!gs_before(p, sm, t.k, t.b, c, live, m0))) break;
    const float2 m_in = gs_carry(sm, t.k, lane);
    if (warp == 0 && live) {
      const float2 out = make_float2(fmaf(At.x, m_in.x, Mt.x), fmaf(At.y, m_in.y, Mt.y));
      if (t.k + 1 == p.tiles) {
        if (p.dh0 != nullptr) *reinterpret_cast<float2*>(p.dh0 + at) = out;
      } else if ((t.k + 1) % kGsGroup == 0) {
        gs_publish(p.group + (t.k + 1) / kGsGroup * step + at, gs_pack(0.f, out.x));
        gs_publish(p.group + (t.k + 1) / kGsGroup * step + at + 1, gs_pack(0.f, out.y));
      }
    }
    float2 m = make_float2(fmaf(Ab.x, m_in.x, Mb.x), fmaf(Ab.y, m_in.y, Mb.y)), db = zero;
#pragma unroll
    for (int r = kGsRun - 1; r >= 0; --r) {
      const float2 dy = gs_load2(&sm.tile[stage][2][warp * kGsRun + r][2 * lane]);
      const float2 l = make_float2(dy.x + m.x, dy.y + m.y);
      float2 a, na;
      gs_split(s[r].x, &a.x, &na.x);
      gs_split(s[r].y, &a.y, &na.y);
      const float2 dg = make_float2(l.x * w[r].x * (a.x * na.x), l.y * w[r].y * (a.y * na.y));
      m = make_float2(a.x * l.x, a.y * l.y);
      const int row = sm.row[stage][warp * kGsRun + r];
      if (row >= 0 && live) {
        const long long o = (long long)t.b * p.n + row;
        gs_store2(static_cast<T_*>(p.dx) + o * p.lddx + c, na.x * l.x, na.y * l.y);
        gs_store2(static_cast<T_*>(p.dg) + o * p.lddg + c, dg.x, dg.y);
        db = make_float2(db.x + dg.x, db.y + dg.y);
      }
    }
    if (p.dbias_part != nullptr) {
      sm.db[warp][lane] = db;
      __syncthreads();
      if (warp == 0 && live) {
        float2 v = zero;
#pragma unroll
        for (int q = 0; q < kGsWarps; ++q) v = make_float2(v.x + sm.db[q][lane].x, v.y + sm.db[q][lane].y);
        *reinterpret_cast<float2*>(p.dbias_part + ((long long)t.b * p.tiles + kr) * p.D + c) = v;
      }
    }
    cur = nxt;
    t = u;
    stage ^= 1;
  }
  cp_async_wait<0>();
}

// dbias [D] = the tiles' partial sums, added in their order (the same result on every run): a block takes 32 channels,
// each of its 32 warps every 32nd part.
__global__ void __launch_bounds__(1024) gated_scan_bias_kernel(const float* __restrict__ part, int parts, int D,
                                                               float* __restrict__ dbias) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int k = warp; k < parts; k += 32) v += part[(long long)k * D + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < D) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s[k][lane];
    dbias[c] = v;
  }
}

}  // namespace mate
