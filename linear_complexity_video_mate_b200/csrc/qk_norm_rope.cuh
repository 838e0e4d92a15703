// Norms of queries and keys for each head with the position rotation in the same pass, and its gradient
// (optional step between the qkv projection and the window attention; the pages describe neither).
//
// Per head vector x[tp] of a q or k head:  r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  z = R y, where R turns
// each channel pair (u, v) by the angle of the token's position along one grid axis:
//   (u, v) -> (u cos - v sin, v cos + u sin).
// Backward: dy = R^T dz,  dw = sum of dy x r over rows and heads,  g = dy w,  dx = r (g - x r mean(g x r)).
//
// Bound by HBM: every value is read and written once.  A warp takes one row at a time.  G lanes (a power of two) share
// a head vector, each with PAIRS channel pairs of it, and 32 / G heads are worked on at a time; a lane has the same
// channels in every head, so the token's cos and sin and the weights of those channels are fetched once per row and
// once per warp.  Both halves of every pair are in one lane: adjacent channels as 16-byte vectors, halves as two
// vectors of half that width, so the rotation needs no exchange; the norm is a sum over G lanes.  2 x 147,456 rows of
// 16 + 16 + 16 heads of 128 bf16 channels: 1.19 ms, 0.93 of the measured copy rate (a warp per row that walked one head
// after another through shared memory took 5.2 ms).
#pragma once
#include "common.cuh"
#include "mamba_extras.cuh"   // to_f32, from_f32

namespace mate {

struct QkParams {
  const void* x;       // [rows, ldx]: q heads | k heads | v heads
  long long ldx;
  const float *wq, *wk;          // [tp] or null
  const float2 *tab_t, *tab_h, *tab_w;   // [T][rt/2], [H][rh/2], [W][rw/2]: (cos, sin)
  void* out;           // forward: z | v; backward: dx | dv
  long long ldo;
  const void* dz;      // backward: gradient of the output
  long long ldz;
  float* part;         // backward: per block [2][tp] partial weight gradients
  long long rows;
  FastDiv n, H, W;     // tokens of a sample, H, W
  int hq, hk, hv, tp;
  int rt, rh, rw;
  int pairing;         // 0: channels 2i, 2i+1 of an axis block; 1: channels i, i + r/2
  float eps;
  int copy_v;
  FastDiv splits;      // warps that share a row's heads
};

constexpr int kQkMaxDim = 256;
constexpr int kQkWarps = 8;
constexpr int kQkMaxParts = 512;     // blocks of the backward pass, with a partial sum of the weight gradients each

// out [cols] = the parts' rows of [parts][cols], added in a fixed order (the same result on every run): a block takes 32
// columns, each of its 32 warps every 32nd part.  Columns from `split` on go to out2; either may be null.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* __restrict__ part, int parts, int cols,
                                                         float* __restrict__ out, int split, float* __restrict__ out2) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int k = warp; k < parts; k += 32) v += part[(long long)k * cols + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s[k][lane];
    if (c < split) {
      if (out != nullptr) out[c] = v;
    } else if (out2 != nullptr) {
      out2[c - split] = v;
    }
  }
}

// How a lane's 16-byte units lie in a head and how their channels pair up.
enum : int {
  kQkAdjacent = 0,   // 16 contiguous bytes; channels 2i, 2i + 1 pair up
  kQkHalves = 1,     // 8 bytes of the first half of an axis' channels and the 8 they pair with (r a multiple of 16 bytes)
  kQkAny = 2         // 16 contiguous bytes, partners through shared memory (halves that 8-byte units do not divide)
};

// Values of one lane: NV units of V channels, as P pairs of fp32 values each.
template <typename T_, int MODE, int NV>
struct QkLane {
  static constexpr int V = 16 / sizeof(T_), P = V / 2, HV = V / 2;
  static constexpr int C = MODE == kQkAny ? V : P;   // (cos, sin) entries per unit
  float2 cs[NV][C];        // the row's cos and sin (kQkHalves: first all cos, then all sin of the unit's pairs)
  int c[NV][2];            // first channel of the unit (kQkHalves: of its two halves)
  int axis[NV][C], idx[NV][C], partner[MODE == kQkAny ? NV : 1][MODE == kQkAny ? V : 1];
  bool on[NV];

  // Axis and table entry of channel c (axis 3: not rotated), and the channel it pairs with.
  static __device__ __forceinline__ int locate(const QkParams& p, int ch, int* i, int* other, bool* second) {
    const int b1 = p.rt, b2 = b1 + p.rh, b3 = b2 + p.rw;
    const int ax = ch < b1 ? 0 : ch < b2 ? 1 : ch < b3 ? 2 : 3;
    const int c0 = ax == 0 ? 0 : ax == 1 ? b1 : ax == 2 ? b2 : b3;
    const int half = (ax == 0 ? p.rt : ax == 1 ? p.rh : ax == 2 ? p.rw : p.tp - b3) / 2, k = ch - c0;
    if (p.pairing == 0) {
      *i = k >> 1;
      *second = k & 1;
      *other = ch ^ 1;
    } else {
      *second = k >= half;
      *i = *second ? k - half : k;
      *other = *second ? ch - half : ch + half;
    }
    if (ax == 3) *other = ch;
    return ax;
  }

  __device__ __forceinline__ void init(const QkParams& p, int e, int G) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int u = e + n * G;
      on[n] = u < p.tp / V;
      int i, o;
      bool s;
      if constexpr (MODE == kQkHalves) {
        // units run over the first halves of the axes' channels, then of the ones that stay
        int left = on[n] ? u * HV : 0, c0 = 0, r = p.rt;
        if (left >= r / 2) { left -= r / 2; c0 += r; r = p.rh; }
        if (c0 == p.rt && r == p.rh && left >= r / 2) { left -= r / 2; c0 += r; r = p.rw; }
        if (c0 == p.rt + p.rh && r == p.rw && left >= r / 2) { left -= r / 2; c0 += r; r = p.tp - c0; }
        c[n][0] = c0 + left;
        c[n][1] = c[n][0] + r / 2;
      } else {
        c[n][0] = on[n] ? u * V : 0;
        c[n][1] = c[n][0] + HV;
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int ch = c[n][0] + (MODE == kQkAdjacent ? 2 * k : k);
        axis[n][k] = locate(p, ch, &i, &o, &s);
        idx[n][k] = i;
        if constexpr (MODE == kQkAny) partner[n][k] = s ? ~o : o;   // the second of a pair, negated
      }
    }
  }

  // First channel of pair k of unit n.
  __device__ __forceinline__ int channel(int n, int k) const { return c[n][2 * k / HV] + 2 * k % HV; }

  // The row's cos and sin of this lane's channels.
  __device__ __forceinline__ void row(const QkParams& p, unsigned row) {
    const unsigned tok = row - p.n.div(row) * p.n.d, rest = p.W.div(tok), wi = tok - rest * p.W.d, ti = p.H.div(rest),
                   hi = rest - ti * p.H.d;
    const float2* t0 = p.tab_t + (long long)ti * (p.rt / 2);
    const float2* t1 = p.tab_h + (long long)hi * (p.rh / 2);
    const float2* t2 = p.tab_w + (long long)wi * (p.rw / 2);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      float2 v[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int ax = axis[n][k];
        v[k] = ax == 3 ? make_float2(1.f, 0.f) : __ldg((ax == 0 ? t0 : ax == 1 ? t1 : t2) + idx[n][k]);
        if constexpr (MODE == kQkAny)
          if (partner[n][k] >= 0) v[k].y = -v[k].y;
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        if constexpr (MODE == kQkHalves)
          cs[n][k] = k < P / 2 ? make_float2(v[2 * k].x, v[2 * k + 1].x)
                               : make_float2(v[2 * (k - P / 2)].y, v[2 * (k - P / 2) + 1].y);
        else
          cs[n][k] = v[k];
      }
    }
  }

  // (plain loads: the output may be the input)
  __device__ __forceinline__ uint4 load(const T_* head, int n) const {
    if constexpr (MODE == kQkHalves) {
      const uint2 a = *reinterpret_cast<const uint2*>(head + c[n][0]);
      const uint2 b = *reinterpret_cast<const uint2*>(head + c[n][1]);
      return make_uint4(a.x, a.y, b.x, b.y);
    } else {
      return *reinterpret_cast<const uint4*>(head + c[n][0]);
    }
  }
  __device__ __forceinline__ void store(T_* head, int n, const float2 (&v)[P]) const {
    uint4 u;
    if constexpr (sizeof(T_) == 2)
      u = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                     pack_bf16x2(v[3].x, v[3].y));
    else
      u = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    if constexpr (MODE == kQkHalves) {
      *reinterpret_cast<uint2*>(head + c[n][0]) = make_uint2(u.x, u.y);
      *reinterpret_cast<uint2*>(head + c[n][1]) = make_uint2(u.z, u.w);
    } else {
      *reinterpret_cast<uint4*>(head + c[n][0]) = u;
    }
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float2 (&v)[P]) {
    if constexpr (sizeof(T_) == 2) {
      v[0] = bf16_pair(u.x);
      v[1] = bf16_pair(u.y);
      v[2] = bf16_pair(u.z);
      v[3] = bf16_pair(u.w);
    } else {
      v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }

  // The rotation (BACK: its transpose) of a head, values of all its lanes at once (buf: the head's tp values of scratch).
  template <bool BACK>
  __device__ __forceinline__ void rotate(float2 (&v)[NV][P], float* buf) const {
    if constexpr (MODE == kQkAdjacent) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const float co = cs[n][k].x, si = BACK ? -cs[n][k].y : cs[n][k].y;
          const float2 a = v[n][k];
          v[n][k] = make_float2(fmaf(a.x, co, -a.y * si), fmaf(a.y, co, a.x * si));
        }
    } else if constexpr (MODE == kQkHalves) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int k = 0; k < P / 2; ++k) {
          const float2 co = cs[n][k], si = cs[n][k + P / 2], ns = make_float2(-si.x, -si.y);
          const float2 a = v[n][k], b = v[n][k + P / 2];
          v[n][k] = fma2(a, co, mul_f32x2(b, BACK ? si : ns));
          v[n][k + P / 2] = fma2(b, co, mul_f32x2(a, BACK ? ns : si));
        }
    } else {
      __syncwarp();   // the head before is read
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (on[n])
#pragma unroll
          for (int k = 0; k < P; ++k) *reinterpret_cast<float2*>(buf + c[n][0] + 2 * k) = v[n][k];
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const int a = partner[n][2 * k], b = partner[n][2 * k + 1];
          const float pa = buf[a < 0 ? ~a : a], pb = buf[b < 0 ? ~b : b];
          const float2 ca = cs[n][2 * k], cb = cs[n][2 * k + 1];
          v[n][k] = make_float2(fmaf(v[n][k].x, ca.x, pa * (BACK ? -ca.y : ca.y)),
                                fmaf(v[n][k].y, cb.x, pb * (BACK ? -cb.y : cb.y)));
        }
    }
  }
};

// Sum over the G lanes of a head.
__device__ __forceinline__ float group_sum(float v, int G) {
  for (int o = G >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Which of a row's heads a warp works on: unit -> row, part.
struct QkUnit {
  int row, part;
  __device__ __forceinline__ QkUnit(const QkParams& p, unsigned u) {
    row = static_cast<int>(p.splits.div(u));
    part = static_cast<int>(u - row * p.splits.d);
  }
};

// Copies the value heads of a row.
template <typename T_>
__device__ __forceinline__ void qk_copy_v(const QkParams& p, const T_* src, T_* dst, int part) {
  constexpr int V = 16 / sizeof(T_);
  const int c0 = (p.hq + p.hk) * p.tp, nv = p.hv * p.tp / V, step = 32 * static_cast<int>(p.splits.d);
  const uint4* s = reinterpret_cast<const uint4*>(src + c0);
  uint4* d = reinterpret_cast<uint4*>(dst + c0);
  for (int v = part * 32 + (threadIdx.x & 31); v < nv; v += 4 * step) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v + j * step < nv) u[j] = s[v + j * step];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v + j * step < nv) d[v + j * step] = u[j];
  }
}

// Eight heads' loads are in flight per warp (four: 1.27 ms for the rows above; three blocks per SM instead of two: 1.38 ms,
// their registers spill).
template <typename T_, int MODE, int NV, int G>
__global__ void __launch_bounds__(kQkWarps * 32, 2) qk_norm_rope_kernel(const QkParams p) {
  using L = QkLane<T_, MODE, NV>;
  constexpr int HPW = 32 / G, UN = NV == 1 ? 8 : 2;   // heads at a time, and how many of those are loaded ahead
  __shared__ float s_buf[MODE == kQkAny ? kQkWarps * 32 * NV * L::V : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G;
  float* buf = s_buf + (MODE == kQkAny ? (warp * HPW + slot) * (G * NV * L::V) : 0);
  const unsigned units = static_cast<unsigned>(p.rows) * p.splits.d;   // below 2^31: rows are shared only where they are few
  const int splits = p.splits.d;
  const float inv_tp = 1.f / p.tp;
  L l;
  l.init(p, lane % G, G);
  float2 wt[2][NV][L::P];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < L::P; ++k) {
        const float* w = q == 0 ? p.wq : p.wk;
        wt[q][n][k] = w != nullptr ? __ldg(reinterpret_cast<const float2*>(w + l.channel(n, k))) : both(1.f);
      }
  for (unsigned u = blockIdx.x * kQkWarps + warp; u < units; u += gridDim.x * kQkWarps) {
    const QkUnit un(p, u);
    l.row(p, un.row);
    const T_* x = static_cast<const T_*>(p.x) + un.row * p.ldx;
    T_* out = static_cast<T_*>(p.out) + un.row * p.ldo;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int h0 = kind == 0 ? 0 : p.hq, h1 = kind == 0 ? p.hq : p.hq + p.hk;
      for (int b = h0 + un.part * HPW + slot; b - slot < h1; b += UN * splits * HPW) {
        uint4 raw[UN][NV];
#pragma unroll
        for (int j = 0; j < UN; ++j) {
          const int head = b + j * splits * HPW;
#pragma unroll
          for (int n = 0; n < NV; ++n)
            raw[j][n] = head < h1 && l.on[n] ? l.load(x + head * p.tp, n) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < UN; ++j) {
          const int head = b + j * splits * HPW;
          if (head - slot >= h1) break;   // the same for the warp
          float2 v[NV][L::P], ss = both(0.f);
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            L::unpack(raw[j][n], v[n]);
#pragma unroll
            for (int k = 0; k < L::P; ++k) ss = fma2(v[n][k], v[n][k], ss);
          }
          const float r = rsqrtf(fmaf(group_sum(ss.x + ss.y, G), inv_tp, p.eps));
#pragma unroll
          for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int k = 0; k < L::P; ++k) v[n][k] = mul_f32x2(mul_f32x2(v[n][k], both(r)), wt[kind][n][k]);
          l.template rotate<false>(v, buf);
          if (head < h1)
#pragma unroll
            for (int n = 0; n < NV; ++n)
              if (l.on[n]) l.store(out + head * p.tp, n, v[n]);
        }
      }
    }
    if (p.copy_v) qk_copy_v(p, x, out, un.part);
  }
}

// The head that a slot of the warp takes in a turn (-1: none).
__device__ __forceinline__ int qk_head(const QkParams& p, int turn, int turns_q, int hpw, int slot) {
  const int q = turn * hpw + slot, k = (turn - turns_q) * hpw + slot;
  return turn < turns_q ? (q < p.hq ? q : -1) : (k < p.hk ? p.hq + k : -1);
}

// The sums of the weight gradients stay in a lane's registers over all its rows.  16,384 rows of 8 + 8 + 8 heads of 64
// bf16 channels: 33 us (half of the copy rate, 16 warps per SM at 128 registers; three blocks per SM spill: 70 us).
template <typename T_, int MODE, int NV, int G>
__global__ void __launch_bounds__(kQkWarps * 32, 2) qk_norm_rope_bwd_kernel(const QkParams p) {
  using L = QkLane<T_, MODE, NV>;
  constexpr int HPW = 32 / G, UN = NV == 1 ? 4 : 1;
  __shared__ float s_buf[MODE == kQkAny ? kQkWarps * 32 * NV * L::V : 1];
  __shared__ float s_dw[kQkWarps][2][kQkMaxDim];
  __shared__ float s_w[2][kQkMaxDim];   // the weights: not in registers, which the loads ahead and the sums need
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G;
  float* buf = s_buf + (MODE == kQkAny ? (warp * HPW + slot) * (G * NV * L::V) : 0);
  const unsigned units = static_cast<unsigned>(p.rows) * p.splits.d;   // below 2^31: rows are shared only where they are few
  const int splits = p.splits.d;
  const float inv_tp = 1.f / p.tp;
  const int turns_q = (p.hq + HPW - 1) / HPW, turns = turns_q + (p.hk + HPW - 1) / HPW;
  for (int i = threadIdx.x; i < 2 * p.tp; i += blockDim.x) {
    const int q = i / p.tp, c = i - q * p.tp;
    const float* w = q == 0 ? p.wq : p.wk;
    s_w[q][c] = w != nullptr ? __ldg(w + c) : 1.f;
  }
  __syncthreads();
  L l;
  l.init(p, lane % G, G);
  float2 dw[2][NV][L::P];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < L::P; ++k) dw[q][n][k] = both(0.f);
  for (unsigned u = blockIdx.x * kQkWarps + warp; u < units; u += gridDim.x * kQkWarps) {
    const QkUnit un(p, u);
    l.row(p, un.row);
    const T_* x = static_cast<const T_*>(p.x) + un.row * p.ldx;
    const T_* dz = static_cast<const T_*>(p.dz) + un.row * p.ldz;
    T_* out = static_cast<T_*>(p.out) + un.row * p.ldo;
    // turns of the warp: the q heads HPW at a time, then the k heads
    for (int b = un.part; b < turns; b += UN * splits) {
      uint4 raw[UN][NV], rawz[UN][NV];
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        const int head = qk_head(p, b + j * splits, turns_q, HPW, slot);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const bool ok = b + j * splits < turns && head >= 0 && l.on[n];
          raw[j][n] = ok ? l.load(x + head * p.tp, n) : make_uint4(0, 0, 0, 0);
          rawz[j][n] = ok ? l.load(dz + head * p.tp, n) : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        if (b + j * splits >= turns) break;
        const int head = qk_head(p, b + j * splits, turns_q, HPW, slot), kind = b + j * splits >= turns_q;
        float2 v[NV][L::P], g[NV][L::P], ss = both(0.f), gx = both(0.f);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          L::unpack(raw[j][n], v[n]);
          L::unpack(rawz[j][n], g[n]);
#pragma unroll
          for (int k = 0; k < L::P; ++k) ss = fma2(v[n][k], v[n][k], ss);
        }
        const float r = rsqrtf(fmaf(group_sum(ss.x + ss.y, G), inv_tp, p.eps));
        l.template rotate<true>(g, buf);
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int k = 0; k < L::P; ++k) {
            v[n][k] = mul_f32x2(v[n][k], both(r));
            if (kind == 0) dw[0][n][k] = fma2(g[n][k], v[n][k], dw[0][n][k]);
            else dw[1][n][k] = fma2(g[n][k], v[n][k], dw[1][n][k]);
            g[n][k] = mul_f32x2(g[n][k], *reinterpret_cast<const float2*>(&s_w[kind][l.channel(n, k)]));
            gx = fma2(g[n][k], v[n][k], gx);
          }
        const float m = -group_sum(gx.x + gx.y, G) * inv_tp;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int k = 0; k < L::P; ++k) g[n][k] = mul_f32x2(fma2(v[n][k], both(m), g[n][k]), both(r));
        if (head >= 0)
#pragma unroll
          for (int n = 0; n < NV; ++n)
            if (l.on[n]) l.store(out + head * p.tp, n, g[n]);
      }
    }
    if (p.copy_v) qk_copy_v(p, dz, out, un.part);
  }
  // the block's weight gradients: the warp's head slots, then the warps, in order
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < L::P; ++k) {
        float2 d = dw[q][n][k];
        for (int o = G; o < 32; o <<= 1) {
          d.x += __shfl_xor_sync(0xffffffffu, d.x, o);
          d.y += __shfl_xor_sync(0xffffffffu, d.y, o);
        }
        if (slot == 0 && l.on[n])
          *reinterpret_cast<float2*>(&s_dw[warp][q][l.channel(n, k)]) = d;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.tp; i += blockDim.x) {
    const int kind = i / p.tp, c = i % p.tp;
    float v = 0.f;
    for (int k = 0; k < kQkWarps; ++k) v += s_dw[k][kind][c];
    p.part[(long long)blockIdx.x * 2 * p.tp + i] = v;
  }
}

// (cos, sin) of (start + p) theta^(-2 i / dims), p < count, i < dims / 2, the angle in 64 bits.
__global__ void __launch_bounds__(256) rope_table_kernel(float2* __restrict__ tab, double start, int count, int half,
                                                         double theta) {
  const long long total = (long long)count * half;
  for (long long k = (long long)blockIdx.x * blockDim.x + threadIdx.x; k < total;
       k += (long long)gridDim.x * blockDim.x) {
    const int i = static_cast<int>(k % half);
    double s, c;
    sincos((start + static_cast<double>(k / half)) * pow(theta, -static_cast<double>(i) / half), &s, &c);
    tab[k] = make_float2(static_cast<float>(c), static_cast<float>(s));
  }
}

}  // namespace mate
