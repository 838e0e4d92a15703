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

// x / s to the nearest integer for |x| <= 127.5 s, decided exactly: the product with 1/s is off by at most
// 127 * 2^-23 < 2^-10, so only quotients that near a midpoint need the remainder x - k s, which one fma gives
// without error there (it has at most as many bits as x).
__device__ __forceinline__ int quant_round(float x, float s, float inv) {
  const float t = x * inv;
  float k = rintf(t);
  if (fabsf(t - k) > 0.4990234375f) {
    const float e2 = 2.f * fmaf(-k, s, x);
    if (e2 > s || (e2 == s && (static_cast<int>(k) & 1))) k += 1.f;
    else if (e2 < -s || (e2 == -s && (static_cast<int>(k) & 1))) k -= 1.f;
  }
  return static_cast<int>(k);
}

constexpr float kQuantTiny = 1e-30f;   // scales below: 1 / s may overflow, the quotient is formed in 64 bits

__device__ __forceinline__ int quant_round_tiny(float x, float s) {
  if (s == 0.f) return 0;   // a row of zeros, or of values whose scale rounds to zero
  return static_cast<int>(fmin(fmax(rint(static_cast<double>(x) / static_cast<double>(s)), -127.0), 127.0));
}

// One warp per row, 16 bytes of q per lane and step.  A row with an infinity or NaN gets scale NaN and q = 0, so
// that the projection of that row is NaN.
template <typename T_>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T_* __restrict__ x, long long ldx, long long M, int K,
                                                            int8_t* __restrict__ q, long long ldq,
                                                            float* __restrict__ scale) {
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  for (long long r = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < M; r += warps) {
    const T_* xr = x + r * ldx;
    unsigned mx = 0;   // |x| as bits: ordered like the values, NaN above infinity
    for (int c = lane; c < K; c += 32) mx = max(mx, __float_as_uint(to_f32(xr[c])) & 0x7fffffffu);
    mx = __reduce_max_sync(0xffffffffu, mx);
    const bool bad = mx >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(mx) / 127.f;
    const float inv = 1.f / s;
    for (int c = lane; c < K; c += 32) {
      const float v = to_f32(xr[c]);
      q[r * ldq + c] = static_cast<int8_t>(bad ? 0 : s < kQuantTiny ? quant_round_tiny(v, s) : quant_round(v, s, inv));
    }
    if (lane == 0) scale[r] = s;
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
  uint64_t* tempty = tfull + 2;           // leader only: both CTAs' epilogues drained the accumulator
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
      mbar_init(&tempty[a], 2 * kI8EpiWarps);
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
    }
  } else {
    const int quad = warp & 3;
    const int chalf = (warp - 2) >> 2;
    int it = 0;
    for (int tile = pair; tile < p.num_tiles; tile += npairs, ++it) {
      const int mb = tile / p.num_n_tiles, nb = tile % p.num_n_tiles;
      const int acc = it & 1;
      const uint32_t acc_par = (it >> 1) & 1;
      if (!mbar_wait(&tfull[acc], acc_par)) break;
      tc_fence_after();
      const int row = mb * 256 + rank * 128 + quad * 32 + lane;
      const bool row_ok = row < p.M;
      const float as = row_ok ? __ldg(p.a_scale + row) : 0.f;
      T_* crow = static_cast<T_*>(p.C) + (long long)row * p.ldc;
      const int cols = min(p.bn, p.N - nb * p.bn);
      for (int c0 = chalf * 32; c0 < cols; c0 += 64) {
        uint32_t r[32];
        tmem_ld32(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256 + c0, r);
        tmem_wait_ld();
        if (row_ok) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int col = nb * p.bn + c0 + j;
            if (c0 + j < cols) {
              float v = static_cast<float>(static_cast<int>(r[j])) * as * __ldg(p.w_scale + col);
              if (p.bias != nullptr) v += __ldg(p.bias + col);
              crow[col] = from_f32<T_>(v);
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_cta(&tempty[acc], 0));
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
