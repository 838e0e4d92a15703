// Norms of queries and keys for each head with the position rotation in the same pass, and its gradient
// (optional step between the qkv projection and the window attention; the pages describe neither).
//
// Per head vector x[tp] of a q or k head:  r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  z = R y, where R turns
// each channel pair (u, v) by the angle of the token's position along one grid axis:
//   (u, v) -> (u cos - v sin, v cos + u sin).
// Backward: dy = R^T dz,  dw = sum of dy x r over rows and heads,  g = dy w,  dx = r (g - x r mean(g x r)).
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
  int T, H, W;
  int hq, hk, hv, tp;
  int rt, rh, rw;
  int pairing;         // 0: channels 2i, 2i+1 of an axis block; 1: channels i, i + r/2
  float eps;
  int copy_v;
};

constexpr int kQkMaxDim = 256;
constexpr int kQkWarps = 8;
constexpr int kQkMaxBlocks = 1184;   // 8 blocks per SM: also the number of partial weight gradients

// The partner of channel c and the (cos, signed sin) of its rotation: z_c = y_c cos + s y_partner sin with
// s = -1 for the pair's first channel, +1 for its second.  Channels behind the rotated ones: (c, 1, 0).
__device__ __forceinline__ void qk_pair(const QkParams& p, int c, int t, int h, int w, int* partner, float* co,
                                        float* si) {
  const float2* tab;
  int r;
  int c0 = 0;
  if (c < p.rt) {
    r = p.rt;
    tab = p.tab_t + (long long)t * (r / 2);
  } else if (c < p.rt + p.rh) {
    c0 = p.rt;
    r = p.rh;
    tab = p.tab_h + (long long)h * (r / 2);
  } else if (c < p.rt + p.rh + p.rw) {
    c0 = p.rt + p.rh;
    r = p.rw;
    tab = p.tab_w + (long long)w * (r / 2);
  } else {
    *partner = c;
    *co = 1.f;
    *si = 0.f;
    return;
  }
  const int i = c - c0;
  const int pi = p.pairing == 0 ? i >> 1 : (i < r / 2 ? i : i - r / 2);
  const bool second = p.pairing == 0 ? (i & 1) : i >= r / 2;
  const float2 cs = __ldg(tab + pi);
  *partner = c0 + (p.pairing == 0 ? (i ^ 1) : (second ? i - r / 2 : i + r / 2));
  *co = cs.x;
  *si = second ? cs.y : -cs.y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp per row; lanes walk the channels of one head after another.
template <typename T_>
__global__ void __launch_bounds__(kQkWarps * 32) qk_norm_rope_kernel(QkParams p) {
  __shared__ float s_y[kQkWarps][kQkMaxDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = p.T * p.H * p.W;
  for (long long row = (long long)blockIdx.x * kQkWarps + warp; row < p.rows; row += (long long)gridDim.x * kQkWarps) {
    const int tok = static_cast<int>(row % n);
    const int w = tok % p.W, h = (tok / p.W) % p.H, t = tok / (p.W * p.H);
    const T_* x = static_cast<const T_*>(p.x) + row * p.ldx;
    T_* out = static_cast<T_*>(p.out) + row * p.ldo;
    for (int head = 0; head < p.hq + p.hk; ++head) {
      const float* wt = head < p.hq ? p.wq : p.wk;
      float ss = 0.f;
      for (int c = lane; c < p.tp; c += 32) {
        const float v = to_f32(x[head * p.tp + c]);
        s_y[warp][c] = v;
        ss = fmaf(v, v, ss);
      }
      const float r = rsqrtf(warp_sum(ss) / p.tp + p.eps);
      for (int c = lane; c < p.tp; c += 32) s_y[warp][c] *= wt != nullptr ? r * wt[c] : r;
      __syncwarp();
      for (int c = lane; c < p.tp; c += 32) {
        int pc;
        float co, si;
        qk_pair(p, c, t, h, w, &pc, &co, &si);
        out[head * p.tp + c] = from_f32<T_>(s_y[warp][c] * co + s_y[warp][pc] * si);
      }
      __syncwarp();
    }
    if (p.copy_v)
      for (int c = (p.hq + p.hk) * p.tp + lane; c < (p.hq + p.hk + p.hv) * p.tp; c += 32) out[c] = x[c];
  }
}

template <typename T_>
__global__ void __launch_bounds__(kQkWarps * 32) qk_norm_rope_bwd_kernel(QkParams p) {
  __shared__ float s_z[kQkWarps][kQkMaxDim];
  __shared__ float s_x[kQkWarps][kQkMaxDim];
  __shared__ float s_dw[kQkWarps][2][kQkMaxDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = p.T * p.H * p.W;
  for (int c = lane; c < 2 * kQkMaxDim; c += 32) (&s_dw[warp][0][0])[c] = 0.f;
  for (long long row = (long long)blockIdx.x * kQkWarps + warp; row < p.rows; row += (long long)gridDim.x * kQkWarps) {
    const int tok = static_cast<int>(row % n);
    const int w = tok % p.W, h = (tok / p.W) % p.H, t = tok / (p.W * p.H);
    const T_* x = static_cast<const T_*>(p.x) + row * p.ldx;
    const T_* dz = static_cast<const T_*>(p.dz) + row * p.ldz;
    T_* out = static_cast<T_*>(p.out) + row * p.ldo;
    for (int head = 0; head < p.hq + p.hk; ++head) {
      const int kind = head < p.hq ? 0 : 1;
      const float* wt = kind == 0 ? p.wq : p.wk;
      float ss = 0.f;
      for (int c = lane; c < p.tp; c += 32) {
        const float v = to_f32(x[head * p.tp + c]);
        s_x[warp][c] = v;
        s_z[warp][c] = to_f32(dz[head * p.tp + c]);
        ss = fmaf(v, v, ss);
      }
      const float r = rsqrtf(warp_sum(ss) / p.tp + p.eps);
      __syncwarp();
      float gx = 0.f;
      float g[kQkMaxDim / 32];
#pragma unroll
      for (int j = 0; j < kQkMaxDim / 32; ++j) {
        const int c = lane + 32 * j;
        g[j] = 0.f;
        if (c < p.tp) {
          int pc;
          float co, si;
          qk_pair(p, c, t, h, w, &pc, &co, &si);
          const float dy = s_z[warp][c] * co - s_z[warp][pc] * si;   // the transposed rotation
          const float nx = s_x[warp][c] * r;
          s_dw[warp][kind][c] += dy * nx;
          g[j] = wt != nullptr ? dy * wt[c] : dy;
          gx = fmaf(g[j], nx, gx);
        }
      }
      const float m = warp_sum(gx) / p.tp;
#pragma unroll
      for (int j = 0; j < kQkMaxDim / 32; ++j) {
        const int c = lane + 32 * j;
        if (c < p.tp) out[head * p.tp + c] = from_f32<T_>(r * (g[j] - s_x[warp][c] * r * m));
      }
      __syncwarp();
    }
    if (p.copy_v)
      for (int c = (p.hq + p.hk) * p.tp + lane; c < (p.hq + p.hk + p.hv) * p.tp; c += 32) out[c] = dz[c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.tp; i += blockDim.x) {
    const int kind = i / p.tp, c = i % p.tp;
    float v = 0.f;
    for (int k = 0; k < kQkWarps; ++k) v += s_dw[k][kind][c];
    p.part[(long long)blockIdx.x * 2 * p.tp + i] = v;
  }
}

// dwq | dwk [tp] = the blocks' partial sums, added in block order (the same result on every run).
__global__ void __launch_bounds__(256) qk_weight_grad_kernel(const float* __restrict__ part, int blocks, int tp,
                                                             float* __restrict__ dwq, float* __restrict__ dwk) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= 2 * tp) return;
  float v = 0.f;
  for (int b = lane; b < blocks; b += 32) v += part[(long long)b * 2 * tp + i];
  v = warp_sum(v);
  float* d = i < tp ? dwq : dwk;
  if (lane == 0 && d != nullptr) d[i < tp ? i : i - tp] = v;
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
