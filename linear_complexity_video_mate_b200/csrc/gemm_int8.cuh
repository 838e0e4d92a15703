// Projection in 8-bit integers: C[M, N] = (A[M, K] W[N, K]^T) a_scale[row] w_scale[col] + bias[col], with A and W
// int8 and one fp32 scale per row of each (token and output channel), and the quantisation of the rows of A.
// Integer products and sums are exact (K < 2^17, so a sum stays below 2^31); only the sum's conversion to fp32,
// the two scales, the bias and the output type round.
#pragma once
#include "common.cuh"
#include "mamba_extras.cuh"   // to_f32, from_f32

namespace mate {

// ---------------------------------------------------------------------------------------------------
// Rows to int8: scale = max|x| / 127 (fp32), q = x / scale to the nearest integer, ties to even.
// ---------------------------------------------------------------------------------------------------

// x / s to the nearest integer k for |x| <= 127.5 s: t = x (1/s) is off by at most 127 * 2^-23 < 2^-15, so rounding t
// (by adding 1.5 * 2^23, which leaves k in the sum's low byte) is right unless t is within 2^-15 of a midpoint.
__device__ __forceinline__ float quant_near(float x, float inv, uint32_t* k) {
  const float t = x * inv;
  const float m = t + 12582912.f;
  *k = __float_as_uint(m);
  return fabsf(t - (m - 12582912.f));   // distance from the integer taken
}
constexpr float kQuantMid = 0.5f - 1.f / 32768;

// The same, decided exactly: the remainder x - k s, which one fma gives without error next to a midpoint (it has at most
// as many bits as x there), ties to even.
__device__ __forceinline__ uint32_t quant_round(float x, float s, float inv) {
  float k = rintf(x * inv);
  const float e2 = 2.f * fmaf(-k, s, x);
  if (e2 > s || (e2 == s && (static_cast<int>(k) & 1))) k += 1.f;
  else if (e2 < -s || (e2 == -s && (static_cast<int>(k) & 1))) k -= 1.f;
  return static_cast<uint32_t>(static_cast<int>(k));
}

constexpr float kQuantTiny = 1e-30f;   // scales below: 1 / s may overflow, the quotient is formed in 64 bits

__device__ __forceinline__ int quant_round_tiny(float x, float s) {
  if (s == 0.f) return 0;   // a row of zeros, or of values whose scale rounds to zero
  return static_cast<int>(fmin(fmax(rint(static_cast<double>(x) / static_cast<double>(s)), -127.0), 127.0));
}

// Four values to four bytes.
__device__ __forceinline__ uint32_t quant_pack(float a, float b, float c, float d, float s, float inv) {
  uint32_t x, y, z, w;
  const float off = fmaxf(fmaxf(quant_near(a, inv, &x), quant_near(b, inv, &y)),
                          fmaxf(quant_near(c, inv, &z), quant_near(d, inv, &w)));
  if (off > kQuantMid) {
    x = quant_round(a, s, inv);
    y = quant_round(b, s, inv);
    z = quant_round(c, s, inv);
    w = quant_round(d, s, inv);
  }
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

constexpr int kQuantHeld = 8;   // 16-byte vectors of a row that a thread holds between its two passes

// G threads per row (a warp, or a block where there are few rows), 16-byte loads.  The first kQuantHeld vectors of a
// thread stay in registers, so that a row of up to G * 128 bytes is read once; the rest is read again (from L2).  A row
// with an infinity or NaN gets scale NaN and q = 0, so that the projection of that row is NaN.
template <typename T_, int G>
__global__ void __launch_bounds__(256, 4) quantize_rows_kernel(const T_* __restrict__ x, long long ldx, long long M, int K,
                                                            int8_t* __restrict__ q, long long ldq,
                                                            float* __restrict__ scale) {
  constexpr int V = 16 / sizeof(T_);
  __shared__ unsigned s_mx[8];
  const int t = threadIdx.x % G, lane = threadIdx.x & 31;
  const int nv = K / V;   // whole vectors; the rest of the row goes value by value
  const long long per = blockDim.x / G;
  for (long long r = blockIdx.x * per + threadIdx.x / G; r < M; r += gridDim.x * per) {
    const T_* xr = x + r * ldx;
    int8_t* qr = q + r * ldq;
    uint4 h[kQuantHeld];
    unsigned mx = 0;   // |x| as bits: ordered like the values, NaN above infinity (bf16: two 16-bit halves, joined below)
    auto take = [&](const uint4& u) {
      if constexpr (sizeof(T_) == 2)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                   __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
      else
        mx = max(mx, max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu)));
    };
#pragma unroll
    for (int j = 0; j < kQuantHeld; ++j)
      if (t + j * G < nv) h[j] = __ldg(reinterpret_cast<const uint4*>(xr) + t + j * G);
#pragma unroll
    for (int j = 0; j < kQuantHeld; ++j)
      if (t + j * G < nv) take(h[j]);
    for (int j = t + kQuantHeld * G; j < nv; j += G) take(__ldg(reinterpret_cast<const uint4*>(xr) + j));
    if constexpr (sizeof(T_) == 2) mx = max(mx << 16, mx & 0xffff0000u);
    for (int c = nv * V + t; c < K; c += G) mx = max(mx, __float_as_uint(to_f32(xr[c])) & 0x7fffffffu);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if constexpr (G > 32) {
      __syncthreads();   // the row before is done with s_mx
      if (lane == 0) s_mx[threadIdx.x >> 5] = mx;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < G / 32; ++w) mx = max(mx, s_mx[w]);
    }
    const bool bad = mx >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(mx) / 127.f;
    if (t == 0) scale[r] = s;
    if (bad || s < kQuantTiny) {   // rare
      for (int c = t; c < K; c += G) qr[c] = static_cast<int8_t>(bad ? 0 : quant_round_tiny(to_f32(xr[c]), s));
      continue;
    }
    const float inv = 1.f / s;
    auto put = [&](int j, const uint4& u) {
      if constexpr (sizeof(T_) == 2) {
        const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
        reinterpret_cast<uint2*>(qr)[j] =
            make_uint2(quant_pack(a.x, a.y, b.x, b.y, s, inv), quant_pack(c.x, c.y, d.x, d.y, s, inv));
      } else {
        reinterpret_cast<uint32_t*>(qr)[j] = quant_pack(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                                        __uint_as_float(u.w), s, inv);
      }
    };
#pragma unroll
    for (int j = 0; j < kQuantHeld; ++j)
      if (t + j * G < nv) put(t + j * G, h[j]);
    for (int j = t + kQuantHeld * G; j < nv; j += G) put(j, __ldg(reinterpret_cast<const uint4*>(xr) + j));
    for (int c = nv * V + t; c < K; c += G) qr[c] = static_cast<int8_t>(quant_round(to_f32(xr[c]), s, inv));
  }
}

// ---------------------------------------------------------------------------------------------------
// Few rows (M <= 8): the weights' bytes bound it.  One warp per kFewCols output channels and all M rows; a lane takes
// 16 bytes of K per step (dp4a), the warp adds the lanes' sums at the end.  The rows of A come from L1.
// ---------------------------------------------------------------------------------------------------
constexpr int kFewRows = 8, kFewCols = 4;

template <typename T_, int MR>
__global__ void __launch_bounds__(128) gemm_int8_few_kernel(const int8_t* __restrict__ A, long long lda,
                                                            const float* __restrict__ a_scale, int M, int K,
                                                            const int8_t* __restrict__ W, long long ldw,
                                                            const float* __restrict__ w_scale, int N,
                                                            const float* __restrict__ bias, T_* __restrict__ C,
                                                            long long ldc) {
  const int lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * kFewCols;
  if (n0 >= N) return;
  int acc[MR][kFewCols];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int c = 0; c < kFewCols; ++c) acc[m][c] = 0;
  const int nv = K / 16;
#pragma unroll 4
  for (int v = lane; v < nv; v += 32) {
    int4 w[kFewCols];
#pragma unroll
    for (int c = 0; c < kFewCols; ++c)   // a column behind N repeats the last one
      w[c] = __ldg(reinterpret_cast<const int4*>(W + static_cast<long long>(min(n0 + c, N - 1)) * ldw) + v);
#pragma unroll
    for (int m = 0; m < MR; ++m)
      if (m < M) {
        const int4 a = __ldg(reinterpret_cast<const int4*>(A + m * lda) + v);
#pragma unroll
        for (int c = 0; c < kFewCols; ++c)
          acc[m][c] = __dp4a(a.x, w[c].x, __dp4a(a.y, w[c].y, __dp4a(a.z, w[c].z, __dp4a(a.w, w[c].w, acc[m][c]))));
      }
  }
  for (int k = nv * 16 + lane; k < K; k += 32)
#pragma unroll
    for (int m = 0; m < MR; ++m)
      if (m < M)
#pragma unroll
        for (int c = 0; c < kFewCols; ++c)
          acc[m][c] += static_cast<int>(A[m * lda + k]) * W[static_cast<long long>(min(n0 + c, N - 1)) * ldw + k];
#pragma unroll
  for (int m = 0; m < MR; ++m)
    if (m < M)
#pragma unroll
      for (int c = 0; c < kFewCols; ++c) {
        const int sum = __reduce_add_sync(0xffffffffu, acc[m][c]);
        const int n = n0 + c;
        if (lane == c && n < N) {
          const float v = static_cast<float>(sum) * __ldg(a_scale + m) * __ldg(w_scale + n);
          C[m * ldc + n] = from_f32<T_>(bias != nullptr ? v + __ldg(bias + n) : v);
        }
      }
}

// ---------------------------------------------------------------------------------------------------
// The product: the two-SM persistent pipeline of gemm_bf16.cuh with int8 operands (kind::i8, int32 accumulators).
// A cluster of 2 CTAs computes a 256 x bn tile; each CTA loads its 128 rows of A and bn/2 rows of W (TMA, 128 bytes
// of K per stage, zeros behind K), the leader issues the MMAs, two TMEM accumulators alternate.
// ---------------------------------------------------------------------------------------------------
struct Int8GemmParams {
  int M, N, K;
  int bn;            // tile N (multiple of 32, <= 256)
  int num_n_tiles, num_tiles;
  int stages;
  const float* a_scale;
  const float* w_scale;
  const float* bias;   // or null
  void* C;
  long long ldc;
  int vec;             // rows of C start on 16 bytes
};

constexpr int kI8BK = 128;                               // bytes of K per stage
constexpr int kI8EpiWarps = 8;
constexpr int kI8Threads = (2 + kI8EpiWarps) * 32;

__host__ __device__ inline uint32_t int8_stage_bytes(int bn) { return 128 * 128 + (bn / 2) * 128; }

// int8 x int8 -> int32, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// Chunk swizzle of the transpose buffers: rows of 4 chunks pair up in 128 bytes, rows of 8 fill them.
template <int CH>
__device__ __forceinline__ int int8_swz(int row) { return CH == 4 ? (row >> 1) & 3 : row & 7; }

template <typename T_>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    gemm_int8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const Int8GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t stage_bytes = int8_stage_bytes(p.bn);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * stage_bytes);
  uint64_t* full = bars;                  // leader only: operands of both CTAs landed
  uint64_t* empty = bars + p.stages;      // both CTAs: the pair MMAs are done with this stage
  uint64_t* tfull = bars + 2 * p.stages;  // both CTAs: accumulator ready
  uint64_t* tempty = tfull + 2;           // the CTA's epilogue drained the accumulator (leader: and the other CTA's)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nk = (p.K + kI8BK - 1) / kI8BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kI8EpiWarps + (leader ? 1 : 0));
    }
    mbar_fence_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int tile = pair; tile < p.num_tiles && ok; tile += npairs) {
        const int mb = tile / p.num_n_tiles, nb = tile % p.num_n_tiles;
        // the pair MMA takes W rows [0, n_mma/2) from each CTA (n_mma: the tile's columns rounded up to 32)
        const int n_mma = min(p.bn, (p.N - nb * p.bn + 31) & ~31);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1)) { ok = false; break; }
          uint8_t* sa = smem + stage * stage_bytes;
          const uint32_t full_leader = map_to_cta(&full[stage], 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * stage_bytes);
          tma_load_2d_pair(&tmA, full_leader, sa, kb * kI8BK, mb * 256 + rank * 128);
          tma_load_2d_pair(&tmB, full_leader, sa + 128 * 128, kb * kI8BK, nb * p.bn + rank * (n_mma / 2));
          if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      uint32_t stage = 0, phase = 0;
      int it = 0;
      bool ok = true;
      for (int tile = pair; tile < p.num_tiles && ok; tile += npairs, ++it) {
        const int acc = it & 1;
        const uint32_t acc_par = (it >> 1) & 1;
        const int nb = tile % p.num_n_tiles;
        const int n_mma = min(p.bn, (p.N - nb * p.bn + 31) & ~31);
        const uint32_t idesc = idesc_s8_s32(256, n_mma);
        if (!mbar_wait(&tempty[acc], acc_par ^ 1)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&full[stage], phase)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * stage_bytes);
          const uint32_t sb = sa + 128 * 128;
#pragma unroll
          for (int k = 0; k < kI8BK / 32; ++k)
            mma_i8_pair(d_tmem, desc_sw128(sa + k * 32, 16, 1024), desc_sw128(sb + k * 32, 16, 1024), idesc,
                        (kb | k) != 0);
          mma_commit_pair(map_to_cta(&empty[stage], 0));
          mma_commit_pair(map_to_cta(&empty[stage], 1));
          if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
        }
        mma_commit_pair(map_to_cta(&tfull[acc], 0));
        mma_commit_pair(map_to_cta(&tfull[acc], 1));
      }
    } else if (lane == 0) {
      // passes the other CTA's drained accumulators on: an arrival on the leader's barrier by the epilogue warps
      // themselves would wait for their stores to reach memory first
      int it = 0;
      for (int tile = pair; tile < p.num_tiles; tile += npairs, ++it) {
        if (!mbar_wait(&tempty[it & 1], (it >> 1) & 1)) break;
        mbar_arrive_cluster(map_to_cta(&tempty[it & 1], 0));
      }
    }
  } else {
    // epilogue warps 2..9 -> TMEM lane quadrants 2, 3, 0, 1, 2, 3, 0, 1; warps 2..5 take the even 32-column slices of a
    // tile, warps 6..9 the odd ones.  A slice of 32 rows passes through a transpose buffer, so that the stores write
    // whole row segments.
    const int quad = warp & 3;
    const int chalf = (warp - 2) >> 2;
    constexpr int CH = 32 * sizeof(T_) / 16;   // 16-byte chunks of a row's slice
    uint4* stg = reinterpret_cast<uint4*>(smem + p.stages * stage_bytes + 256) + (warp - 2) * 32 * CH;
    // the column scales and biases of the warp's slices, [4][32] each, fetched while the accumulator fills
    float* sc = reinterpret_cast<float*>(smem + p.stages * stage_bytes + 256 + kI8EpiWarps * 512 * CH) + (warp - 2) * 256;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + chalf * 32;
    int it = 0;
    for (int tile = pair; tile < p.num_tiles; tile += npairs, ++it) {
      const int mb = tile / p.num_n_tiles, nb = tile % p.num_n_tiles;
      const int acc = it & 1;
      const uint32_t acc_par = (it >> 1) & 1;
      const int row0 = mb * 256 + rank * 128 + quad * 32;
      const float as = row0 + lane < p.M ? __ldg(p.a_scale + row0 + lane) : 0.f;
      const int cols = min(p.bn, p.N - nb * p.bn) - chalf * 32;   // of the tile, from this warp's first slice on
      const int first = nb * p.bn + chalf * 32;
      // this lane's chunk of the first 32 / CH rows of a slice, and how far the next rows are
      T_* c_lane = static_cast<T_*>(p.C) + (row0 + lane / CH) * p.ldc + (lane % CH) * (16 / sizeof(T_));
      const long long step = p.ldc * static_cast<long long>(sizeof(T_)) / 16 * (32 / CH);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = i * 64 + lane;
        sc[i * 32 + lane] = c < cols ? __ldg(p.w_scale + first + c) : 0.f;
        sc[128 + i * 32 + lane] = c < cols && p.bias != nullptr ? __ldg(p.bias + first + c) : 0.f;
      }
      __syncwarp();
      if (!mbar_wait(&tfull[acc], acc_par)) break;
      tc_fence_after();
      uint32_t r[32];
      if (cols > 0) {
        tmem_ld32(t_lane + acc * 256, r);
        tmem_wait_ld();
      }
      for (int i = 0; i * 64 < cols; ++i) {
        const int col0 = first + i * 64, left = min(32, cols - i * 64);   // the same for the whole warp
        float2 v[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {   // (acc a_scale) w_scale + bias
          const float4 ws = reinterpret_cast<const float4*>(sc + i * 32)[q];
          const float4 bq = reinterpret_cast<const float4*>(sc + 128 + i * 32)[q];
          const float2 lo = make_float2(static_cast<int>(r[4 * q]), static_cast<int>(r[4 * q + 1]));
          const float2 hi = make_float2(static_cast<int>(r[4 * q + 2]), static_cast<int>(r[4 * q + 3]));
          v[2 * q] = fma2(mul_f32x2(lo, both(as)), make_float2(ws.x, ws.y), make_float2(bq.x, bq.y));
          v[2 * q + 1] = fma2(mul_f32x2(hi, both(as)), make_float2(ws.z, ws.w), make_float2(bq.z, bq.w));
        }
        const bool more = (i + 1) * 64 < cols;
        if (more) {
          tmem_ld32(t_lane + acc * 256 + (i + 1) * 64, r);   // the next slice, while this one is stored
        } else {   // the last one is in registers: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        // row `lane`, chunk q at q ^ (a function of the row): conflict-free both ways
#pragma unroll
        for (int q = 0; q < CH; ++q) {
          uint4 pk;
          if constexpr (sizeof(T_) == 2)
            pk = make_uint4(pack_bf16x2(v[q * 4].x, v[q * 4].y), pack_bf16x2(v[q * 4 + 1].x, v[q * 4 + 1].y),
                            pack_bf16x2(v[q * 4 + 2].x, v[q * 4 + 2].y), pack_bf16x2(v[q * 4 + 3].x, v[q * 4 + 3].y));
          else
            pk = make_uint4(__float_as_uint(v[q * 2].x), __float_as_uint(v[q * 2].y), __float_as_uint(v[q * 2 + 1].x),
                            __float_as_uint(v[q * 2 + 1].y));
          stg[lane * CH + (q ^ int8_swz<CH>(lane))] = pk;
        }
        __syncwarp();
        if (p.vec && left == 32) {
          uint4* dst = reinterpret_cast<uint4*>(c_lane + col0);
#pragma unroll
          for (int j = 0; j < CH; ++j, dst += step) {
            const int rr = j * (32 / CH) + lane / CH;
            if (row0 + rr < p.M) *dst = stg[rr * CH + ((lane % CH) ^ int8_swz<CH>(rr))];
          }
        } else {   // rows of C that do not start on 16 bytes, and the last columns: lane = column
          constexpr int E = 16 / sizeof(T_);
          const int rows = min(32, p.M - row0);
          for (int rr = 0; rr < rows; ++rr)
            if (lane < left)
              (static_cast<T_*>(p.C) + (row0 + rr) * p.ldc + col0)[lane] =
                  reinterpret_cast<const T_*>(stg + rr * CH + ((lane / E) ^ int8_swz<CH>(rr)))[lane % E];
        }
        if (more) tmem_wait_ld();
        __syncwarp();
      }
      if (cols <= 0) {   // a narrow last tile has no slice for these warps
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the leader's MMAs read this CTA's shared memory: nobody leaves before both are done
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace mate
