// Gated linear recurrence over the grid's tokens in one of the four scan orders, and its backward pass (an
// elementwise-state companion of the selective scan; the pages describe only the latter).  Per sample and channel:
//   a_t = sigmoid(g_t + bias),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  y_t = h_t            (h_0 given or zero)
// Backward, with the adjoint state l_t = dy_t + a_{t+1} l_{t+1} (behind the last row: the gradient of h_last):
//   dx_t = (1 - a_t) l_t,  dg_t = l_t (h_{t-1} - x_t) a_t (1 - a_t),  dbias = sum of dg,  dh0 = a_1 l_1.
// States, gates and sums are fp32; y, dx and dg are rounded once on the way out.
#pragma once
#include "common.cuh"
#include "mamba_extras.cuh"   // to_f32, from_f32

namespace mate {

constexpr int kGsChunk = 64;   // rows per saved state: the forward's `states` hold the state before each chunk

struct GatedScanParams {
  const void *x, *g;       // rows b*n + raster, strides ldx, ldg
  long long ldx, ldg;
  const float* bias;       // [D] or null
  const float* h0;         // [B][D] or null
  void* y;                 // forward
  long long ldy;
  float* h_last;           // [B][D] or null
  float* states;           // forward: [B][chunks][D] out or null; backward: in
  const void* dy;          // backward
  long long lddy;
  const float* dh_last;    // [B][D] or null
  void *dx, *dg;
  long long lddx, lddg;
  float* dh0;              // [B][D] or null
  float* dbias_part;       // [B][D] partial sums, or null
  int B, T, H, W, D;
  int order, reverse;
};

// Grid row of step s of the recurrence.
__device__ __forceinline__ long long gs_row(const GatedScanParams& p, int n, int b, int s) {
  return (long long)b * n + scan_to_raster(p.reverse ? n - 1 - s : s, p.T, p.H, p.W, p.order);
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

// One thread per (sample, channel), one step after the other.
template <typename T_>
__global__ void __launch_bounds__(256) gated_scan_kernel(GatedScanParams p) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (c >= p.D) return;
  const int n = p.T * p.H * p.W, chunks = (n + kGsChunk - 1) / kGsChunk;
  const float bias = p.bias != nullptr ? p.bias[c] : 0.f;
  float h = p.h0 != nullptr ? p.h0[(long long)b * p.D + c] : 0.f;
  for (int s = 0; s < n; ++s) {
    if (p.states != nullptr && s % kGsChunk == 0) p.states[((long long)b * chunks + s / kGsChunk) * p.D + c] = h;
    const long long row = gs_row(p, n, b, s);
    const float z = to_f32(static_cast<const T_*>(p.g)[row * p.ldg + c]) + bias;
    h = sigmoid_f(z) * h + sigmoid_f(-z) * to_f32(static_cast<const T_*>(p.x)[row * p.ldx + c]);
    static_cast<T_*>(p.y)[row * p.ldy + c] = from_f32<T_>(h);
  }
  if (p.h_last != nullptr) p.h_last[(long long)b * p.D + c] = h;
}

// One thread per (sample, channel): chunks from the last to the first, each chunk's states formed again from the
// state before it.
template <typename T_>
__global__ void __launch_bounds__(64) gated_scan_bwd_kernel(GatedScanParams p) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (c >= p.D) return;
  const int n = p.T * p.H * p.W, chunks = (n + kGsChunk - 1) / kGsChunk;
  const float bias = p.bias != nullptr ? p.bias[c] : 0.f;
  float lam = p.dh_last != nullptr ? p.dh_last[(long long)b * p.D + c] : 0.f;   // a_{t+1} l_{t+1}
  float db = 0.f;
  float hp[kGsChunk];   // the state before each row of the chunk
  for (int k = chunks - 1; k >= 0; --k) {
    const int s0 = k * kGsChunk, m = min(kGsChunk, n - s0);
    float h = p.states[((long long)b * chunks + k) * p.D + c];
    for (int i = 0; i < m; ++i) {
      hp[i] = h;
      const long long row = gs_row(p, n, b, s0 + i);
      const float z = to_f32(static_cast<const T_*>(p.g)[row * p.ldg + c]) + bias;
      h = sigmoid_f(z) * h + sigmoid_f(-z) * to_f32(static_cast<const T_*>(p.x)[row * p.ldx + c]);
    }
    for (int i = m - 1; i >= 0; --i) {
      const long long row = gs_row(p, n, b, s0 + i);
      const float z = to_f32(static_cast<const T_*>(p.g)[row * p.ldg + c]) + bias;
      const float a = sigmoid_f(z), na = sigmoid_f(-z);
      const float l = to_f32(static_cast<const T_*>(p.dy)[row * p.lddy + c]) + lam;
      const float dg = l * (hp[i] - to_f32(static_cast<const T_*>(p.x)[row * p.ldx + c])) * a * na;
      static_cast<T_*>(p.dx)[row * p.lddx + c] = from_f32<T_>(na * l);
      static_cast<T_*>(p.dg)[row * p.lddg + c] = from_f32<T_>(dg);
      db += dg;
      lam = a * l;
    }
  }
  if (p.dh0 != nullptr) p.dh0[(long long)b * p.D + c] = lam;
  if (p.dbias_part != nullptr) p.dbias_part[(long long)b * p.D + c] = db;
}

// dbias [D] = the partial sums, added in their order (the same result on every run).
__global__ void __launch_bounds__(256) gated_scan_bias_kernel(const float* __restrict__ part, int parts, int D,
                                                              float* __restrict__ dbias) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= D) return;
  float v = 0.f;
  for (int k = 0; k < parts; ++k) v += part[(long long)k * D + c];
  dbias[c] = v;
}

}  // namespace mate
