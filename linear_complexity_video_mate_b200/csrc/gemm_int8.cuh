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

// x / s to the nearest integer k, ties to even, for two |x| <= 127.5 s, exactly.  t = x (1/s) is off by at most
// 127 * 2^-23, so k from t (by adding 1.5 * 2^23, which leaves k in the sum's low byte) is right or the neighbour of the
// right one; the remainder x - k s, which one fma gives without error (it has at most as many bits as x where k is in
// doubt), tells: beyond s / 2, k is one off.  Where the remainder is just s / 2, t decides alone: TIES looks at those, too.
// bf16 rows never need that.  A bf16 x is (k + 1/2) s only if s has at most 8 significant bits; s is the row's maximum, an
// integer p of 8 bits times 2^e, over 127, and p / 127 lies within 2^-24 of such a number only for p = 127 and 254: a power
// of two, whose reciprocal, and with it t, is exact.  Quotients near midpoints are common there (x and the row's maximum
// are ratios of small integers), so the correction has no branch.
template <bool TIES>
__device__ __forceinline__ float2 quant_two(float2 x, float inv, float s, float hs) {
  float2 m = add2(mul_f32x2(x, both(inv)), both(12582912.f));
  const float2 e = fma2(add2(m, both(-12582912.f)), both(-s), x);
  bool px = fabsf(e.x) > hs, py = fabsf(e.y) > hs;
  if (TIES) {
    px = px || (fabsf(e.x) == hs && (__float_as_uint(m.x) & 1u));
    py = py || (fabsf(e.y) == hs && (__float_as_uint(m.y) & 1u));
  }
  if (px) m.x += copysignf(1.f, e.x);
  if (py) m.y += copysignf(1.f, e.y);
  return m;
}
__device__ __forceinline__ uint32_t quant_bytes(float2 lo, float2 hi) {
  return __byte_perm(__byte_perm(__float_as_uint(lo.x), __float_as_uint(lo.y), 0x0040),
                     __byte_perm(__float_as_uint(hi.x), __float_as_uint(hi.y), 0x0040), 0x5410);
}
__device__ __forceinline__ int8_t quant_one(float x, float inv, float s, float hs) {
  return static_cast<int8_t>(__float_as_uint(quant_two<true>(make_float2(x, 0.f), inv, s, hs).x));
}
constexpr float kQuantTiny = 1e-30f;   // scales below: 1 / s may overflow, the quotient is formed in 64 bits

__device__ __forceinline__ int quant_round_tiny(float x, float s) {
  if (s == 0.f) return 0;   // a row of zeros, or of values whose scale rounds to zero
  return static_cast<int>(fmin(fmax(rint(static_cast<double>(x) / static_cast<double>(s)), -127.0), 127.0));
}

// The larger magnitude (NaN if either is one; the sign means nothing), of two packed bf16 or of an fp32 value.
template <typename T_>
__device__ __forceinline__ uint32_t quant_max(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (sizeof(T_) == 2) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("{\n .reg .f32 x, y, z;\n mov.b32 x, %1;\n mov.b32 y, %2;\n max.NaN.xorsign.abs.f32 z, x, y;\n mov.b32 %0, z;\n}"
           : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A row's 16 bytes j, quantised and stored.
template <typename T_>
__device__ __forceinline__ void quant_put(int8_t* qr, int j, const uint4& u, float inv, float s, float hs) {
  if constexpr (sizeof(T_) == 2) {
    const float2 a = quant_two<false>(bf16_pair(u.x), inv, s, hs), b = quant_two<false>(bf16_pair(u.y), inv, s, hs);
    const float2 c = quant_two<false>(bf16_pair(u.z), inv, s, hs), d = quant_two<false>(bf16_pair(u.w), inv, s, hs);
    reinterpret_cast<uint2*>(qr)[j] = make_uint2(quant_bytes(a, b), quant_bytes(c, d));
  } else {
    const float2 a = quant_two<true>(make_float2(__uint_as_float(u.x), __uint_as_float(u.y)), inv, s, hs);
    const float2 b = quant_two<true>(make_float2(__uint_as_float(u.z), __uint_as_float(u.w)), inv, s, hs);
    reinterpret_cast<uint32_t*>(qr)[j] = quant_bytes(a, b);
  }
}

// G threads per row (a warp, or a block where there are few rows or long ones), 16-byte loads.  NV > 0: a thread holds
// the row's NV vectors t, t + G, .. between the two passes, so that the row is read once; NV = 0: rows of any length, read
// twice (the second time from L2).  A row with an infinity or NaN gets scale NaN and q = 0, so that the projection of that
// row is NaN.  262,144 rows of 1024 bf16 values: 139 us, 0.88 of the measured copy rate.
template <typename T_, int G, int NV>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T_* __restrict__ x, long long ldx, int M, int K,
                                                            int8_t* __restrict__ q, long long ldq,
                                                            float* __restrict__ scale) {
  constexpr int V = 16 / sizeof(T_);
  __shared__ uint32_t s_mx[8];
  const int t = threadIdx.x % G, lane = threadIdx.x & 31;
  const int nv = K / V;   // whole vectors; the rest of the row goes value by value
  const int per = 256 / G, step = gridDim.x * per;
  for (int r = blockIdx.x * per + threadIdx.x / G; r < M; r += step) {
    const T_* xr = x + r * ldx;
    const uint4* xv = reinterpret_cast<const uint4*>(xr);
    int8_t* qr = q + r * ldq;
    uint4 h[NV > 0 ? NV : 1];
    uint32_t mx = 0;   // magnitudes as bits (bf16: two at a time): ordered like the values, NaN above infinity
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) h[j] = t + j * G < nv ? __ldg(xv + t + j * G) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        mx = quant_max<T_>(mx, quant_max<T_>(quant_max<T_>(h[j].x, h[j].y), quant_max<T_>(h[j].z, h[j].w)));
    } else {
#pragma unroll 4
      for (int j = t; j < nv; j += G) {
        const uint4 u = __ldg(xv + j);
        mx = quant_max<T_>(mx, quant_max<T_>(quant_max<T_>(u.x, u.y), quant_max<T_>(u.z, u.w)));
      }
    }
    if constexpr (sizeof(T_) == 2) mx = max((mx << 16) & 0x7fffffffu, mx & 0x7fff0000u);
    else mx &= 0x7fffffffu;
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
    const float inv = 1.f / s, hs = 0.5f * s;
    if (bad || s < kQuantTiny) {   // rare
#pragma unroll 1
      for (int c = t; c < K; c += G) {
        const float v = to_f32(xr[c]);
        qr[c] = bad ? 0 : static_cast<int8_t>(quant_round_tiny(v, s));
      }
      continue;
    }
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (t + j * G < nv) quant_put<T_>(qr, t + j * G, h[j], inv, s, hs);
    } else {
      for (int j = t; j < nv; j += G) quant_put<T_>(qr, j, __ldg(xv + j), inv, s, hs);
    }
    for (int c = nv * V + t; c < K; c += G) qr[c] = quant_one(to_f32(xr[c]), inv, s, hs);
  }
}

// ---------------------------------------------------------------------------------------------------
// Few rows: the weights' bytes bound it.  One warp per kFewCols output channels and all M rows; a lane takes
// 16 bytes of K per step (dp4a), the warp adds the lanes' sums at the end.  The rows of A come from L1.
// ---------------------------------------------------------------------------------------------------
// 4096 x 1024 weights, 4 rows: 4.9 us, by the tensor cores 6.9; 12288 x 2048, 2 rows: 8.0 and 12.4; 4 rows: 12.3 and 12.4.
constexpr int kFewRows = 4, kFewCols = 4;

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
//
// An MMA takes 128 cycles (256 x 256 x 32) and reads 8 KB of each CTA's shared memory meanwhile, half of what that
// memory gives; the loads of a stage write as much again, and the epilogue stages its output there too.  So shared
// memory is what bounds the product at short K, and both sides are kept low:
//   KEEP: for K <= kI8KeepK (fp32 output: kI8KeepKF32) a CTA's half of a column tile of W stays in shared memory while the pair walks down the
//   rows, so that only A streams;
//   the epilogue writes a slice of the output to shared memory once and a TMA store takes it from there.
// 262,144 x 1024 x 4368: 0.87 ms, 2.7 Poperations/s, tensor pipe 67% active (without the two: 1.08 ms, 53%);
// 16384 x 4096 x 4096: 3.1 Poperations/s.
// ---------------------------------------------------------------------------------------------------
struct Int8GemmParams {
  int M, N, K;
  int bn;              // tile N (multiple of 32, <= 256)
  int num_n_tiles, num_tiles;
  int stages;
  int slots, groups;   // KEEP: column tiles worked on at a time, pairs per column tile
  const float* a_scale;
  const float* w_scale;
  const float* bias;   // or null
  void* C;
  long long ldc;
  int vec;             // every row of C starts on 16 bytes: TMA stores
};

struct Int8Maps {
  CUtensorMap a, w, c;
};

constexpr int kI8BK = 128;                               // bytes of K per stage
constexpr int kI8KeepK = 1024, kI8KeepKF32 = 768;
constexpr int kI8TileStart = 32;   // what a tile costs beside its columns, in columns (small problems)
constexpr int kI8EpiWarps = 8;
constexpr int kI8Threads = (2 + kI8EpiWarps) * 32;

__host__ __device__ inline uint32_t int8_stage_bytes(int bn, bool keep) {
  return 128 * 128 + (keep ? 0 : (bn / 2) * 128);
}
__host__ __device__ inline uint32_t int8_kept_bytes(int bn, int K, bool keep) {
  return keep ? (K + kI8BK - 1) / kI8BK * (bn / 2) * 128 : 0;
}
// Behind the ring: a 32 x 32 output slice per epilogue warp (1 KB aligned), 256 bytes of barriers, and per epilogue warp
// the scales and biases of its four slices.
__host__ __device__ inline uint32_t int8_out_bytes(int es) { return kI8EpiWarps * 32 * 32 * es; }
constexpr uint32_t kI8Behind = 256 + kI8EpiWarps * 1024;

// The tiles of a pair in order.  KEEP: all rows of a column tile (every groups-th), then its next column tile, so that
// the pairs on different columns read the same rows of A at about the same time.  Else tiles pair, pair + pairs, ...
// with the columns fastest.
template <bool KEEP>
struct Int8Walk {
  int mb, nb, tile, step, mblocks;
  __device__ __forceinline__ Int8Walk(const Int8GemmParams& p, int pair, int npairs) {
    if constexpr (KEEP) {
      mblocks = (p.M + 255) / 256;
      nb = pair % p.slots;
      mb = tile = pair / p.slots;   // its first row tile
      step = p.groups;
    } else {
      tile = pair;
      step = npairs;
      set(p);
    }
  }
  __device__ __forceinline__ void set(const Int8GemmParams& p) {
    mb = tile / p.num_n_tiles;
    nb = tile - mb * p.num_n_tiles;
  }
  __device__ __forceinline__ bool done(const Int8GemmParams& p) const {
    if constexpr (KEEP) return nb >= p.num_n_tiles || tile >= mblocks;
    else return tile >= p.num_tiles;
  }
  __device__ __forceinline__ bool column_starts() const { return KEEP && mb == tile; }
  __device__ __forceinline__ bool column_ends() const { return KEEP && mb + step >= mblocks; }
  __device__ __forceinline__ void next(const Int8GemmParams& p) {
    if constexpr (KEEP) {
      mb += step;
      if (mb >= mblocks) {
        mb = tile;
        nb += p.slots;
      }
    } else {
      tile += step;
      set(p);
    }
  }
};

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

// Arrives once on the barrier at this shared-memory offset in both CTAs of the pair when the pair MMAs issued so far
// have completed.
__device__ __forceinline__ void mma_commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Tiled store from this CTA's shared memory (rows behind the matrix are left out); one thread issues it, and the source
// may be written again once tma_store_read() returns there.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(smem_u32(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Chunk swizzle of a staged slice: rows of 4 chunks (the map's 64-byte swizzle) or 8 (its 128-byte swizzle).
template <int CH>
__device__ __forceinline__ int int8_swz(int row) { return CH == 4 ? (row >> 1) & 3 : row & 7; }

template <typename T_, bool KEEP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    gemm_int8_pair_kernel(const __grid_constant__ Int8Maps maps, const Int8GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t stage_bytes = int8_stage_bytes(p.bn, KEEP);
  uint8_t* kept = smem;                                  // KEEP: W rows of the column tile, 128 bytes of K per block
  uint8_t* ring = smem + int8_kept_bytes(p.bn, p.K, KEEP);
  uint8_t* out = ring + p.stages * stage_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(out + int8_out_bytes(sizeof(T_)));
  uint64_t* full = bars;                  // leader only: operands of both CTAs landed
  uint64_t* empty = bars + p.stages;      // both CTAs: the pair MMAs are done with this stage
  uint64_t* tfull = bars + 2 * p.stages;  // both CTAs: accumulator ready
  uint64_t* tempty = tfull + 2;           // the CTA's epilogue drained the accumulator (leader: and the other CTA's)
  uint64_t* kfull = tempty + 2;           // KEEP, leader only: W rows of the column tile landed
  uint64_t* kempty = kfull + 1;           // KEEP, both CTAs: the pair MMAs are done with them
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kempty + 1);

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
    mbar_init(kfull, 1);
    mbar_init(kempty, 1);
    mbar_fence_init();
    prefetch_tensormap(&maps.a);
    prefetch_tensormap(&maps.w);
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
      uint32_t stage = 0, phase = 0, kphase = 0;
      bool ok = true;
      for (Int8Walk<KEEP> w(p, pair, npairs); ok && !w.done(p); w.next(p)) {
        // the pair MMA takes W rows [0, n_mma/2) from each CTA (n_mma: the tile's columns rounded up to 32)
        const int n_mma = min(p.bn, (p.N - w.nb * p.bn + 31) & ~31);
        const int row_w = w.nb * p.bn + rank * (n_mma / 2);
        if (w.column_starts()) {
          if (!mbar_wait(kempty, kphase ^ 1)) { ok = false; break; }
          kphase ^= 1;
          if (leader) mbar_arrive_expect_tx(kfull, 2 * nk * (p.bn / 2) * 128);
          for (int kb = 0; kb < nk; ++kb)
            tma_load_2d_pair(&maps.w, map_to_cta(kfull, 0), kept + kb * (p.bn / 2) * 128, kb * kI8BK, row_w);
        }
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1)) { ok = false; break; }
          uint8_t* sa = ring + stage * stage_bytes;
          const uint32_t full_leader = map_to_cta(&full[stage], 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * stage_bytes);
          tma_load_2d_pair(&maps.a, full_leader, sa, kb * kI8BK, w.mb * 256 + rank * 128);
          if (!KEEP) tma_load_2d_pair(&maps.w, full_leader, sa + 128 * 128, kb * kI8BK, row_w);
          if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
        }
      }
      // the last arrivals of every stage and of the kept columns come from the leader's commits, in this CTA's shared
      // memory: it does not leave before they are in (a stage or columns never used: the wait passes at once)
      for (int s = 0; ok && s < p.stages; ++s) {
        ok = mbar_wait(&empty[stage], phase ^ 1);
        if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
      }
      if (KEEP && ok) mbar_wait(kempty, kphase ^ 1);
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      uint32_t stage = 0, phase = 0, kphase = 0;
      const uint64_t ring_desc = desc_sw128(smem_u32(ring), 16, 1024), kept_desc = desc_sw128(smem_u32(kept), 16, 1024);
      int it = 0;
      bool ok = true;
      for (Int8Walk<KEEP> w(p, pair, npairs); ok && !w.done(p); w.next(p), ++it) {
        const int acc = it & 1;
        const uint32_t acc_par = (it >> 1) & 1;
        const int n_mma = min(p.bn, (p.N - w.nb * p.bn + 31) & ~31);
        const uint32_t idesc = idesc_s8_s32(256, n_mma);
        if (w.column_starts()) {
          if (!mbar_wait(kfull, kphase)) break;
          kphase ^= 1;
        }
        if (!mbar_wait(&tempty[acc], acc_par ^ 1)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&full[stage], phase)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = ring_desc + stage * (stage_bytes >> 4);
          const uint64_t db = KEEP ? kept_desc + kb * ((p.bn / 2) * 128 >> 4) : da + (128 * 128 >> 4);
#pragma unroll
          for (int k = 0; k < kI8BK / 32; ++k)   // 32 bytes of K further: 2 in the descriptor's 16-byte address units
            mma_i8_pair(d_tmem, da + 2 * k, db + 2 * k, idesc, (kb | k) != 0);
          mma_commit_both(&empty[stage]);
          if (++stage == (uint32_t)p.stages) { stage = 0; phase ^= 1; }
        }
        mma_commit_both(&tfull[acc]);
        if (w.column_ends()) mma_commit_both(kempty);
      }
    } else if (lane == 0) {
      // passes the other CTA's drained accumulators on: an arrival on the leader's barrier by the epilogue warps
      // themselves would wait for their stores to reach memory first
      int it = 0;
      for (Int8Walk<KEEP> w(p, pair, npairs); !w.done(p); w.next(p), ++it) {
        if (!mbar_wait(&tempty[it & 1], (it >> 1) & 1)) break;
        mbar_arrive_cluster(map_to_cta(&tempty[it & 1], 0));
      }
    }
  } else {
    // epilogue warps 2..9 -> TMEM lane quadrants 2, 3, 0, 1, 2, 3, 0, 1; warps 2..5 take the even 32-column slices of a
    // tile, warps 6..9 the odd ones
    const int quad = warp & 3;
    const int chalf = (warp - 2) >> 2;
    constexpr int CH = 32 * sizeof(T_) / 16;   // 16-byte chunks of a row's slice
    uint4* stg = reinterpret_cast<uint4*>(out) + (warp - 2) * 32 * CH;
    float* sc = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 256) + (warp - 2) * 256;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + chalf * 32;
    const bool has_bias = p.bias != nullptr;
    int it = 0;
    for (Int8Walk<KEEP> w(p, pair, npairs); !w.done(p); w.next(p), ++it) {
      const int acc = it & 1;
      const uint32_t acc_par = (it >> 1) & 1;
      const int row0 = w.mb * 256 + rank * 128 + quad * 32;
      const float as = row0 + lane < p.M ? __ldg(p.a_scale + row0 + lane) : 0.f;
      const int cols = min(p.bn, p.N - w.nb * p.bn) - chalf * 32;   // of the tile, from this warp's first slice on
      const int first = w.nb * p.bn + chalf * 32;
      if (!KEEP || w.column_starts()) {   // the column scales and biases of the warp's slices, [4][32] each
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = i * 64 + lane;
          sc[i * 32 + lane] = c < cols ? __ldg(p.w_scale + first + c) : 0.f;
          if (has_bias) sc[128 + i * 32 + lane] = c < cols ? __ldg(p.bias + first + c) : 0.f;
        }
        __syncwarp();
      }
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
        for (int q = 0; q < 8; ++q) {   // (acc a_scale) w_scale
          const float4 ws = reinterpret_cast<const float4*>(sc + i * 32)[q];
          const float2 lo = make_float2(static_cast<int>(r[4 * q]), static_cast<int>(r[4 * q + 1]));
          const float2 hi = make_float2(static_cast<int>(r[4 * q + 2]), static_cast<int>(r[4 * q + 3]));
          v[2 * q] = mul_f32x2(mul_f32x2(lo, both(as)), make_float2(ws.x, ws.y));
          v[2 * q + 1] = mul_f32x2(mul_f32x2(hi, both(as)), make_float2(ws.z, ws.w));
        }
        const bool more = (i + 1) * 64 < cols;
        if (more) {
          tmem_ld32(t_lane + acc * 256 + (i + 1) * 64, r);   // the next slice, while this one is stored
        } else {   // the last one is in registers: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        if (has_bias) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 bq = reinterpret_cast<const float4*>(sc + 128 + i * 32)[q];
            v[2 * q] = add2(v[2 * q], make_float2(bq.x, bq.y));
            v[2 * q + 1] = add2(v[2 * q + 1], make_float2(bq.z, bq.w));
          }
        }
        if (lane == 0) tma_store_read();   // the slice before has left the staging rows
        __syncwarp();
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
        if (p.vec && left == 32) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0 && row0 < p.M) tma_store_2d(&maps.c, stg, col0, row0);
        } else {   // rows of C that do not start on 16 bytes, and the last columns (a store ends at 16 bytes): lane = column
          __syncwarp();
          constexpr int E = 16 / sizeof(T_);
          const int rows = min(32, p.M - row0);
          for (int rr = 0; rr < rows; ++rr)
            if (lane < left)
              (static_cast<T_*>(p.C) + (row0 + rr) * p.ldc + col0)[lane] =
                  reinterpret_cast<const T_*>(stg + rr * CH + ((lane / E) ^ int8_swz<CH>(rr)))[lane % E];
          __syncwarp();
        }
        if (more) tmem_wait_ld();
      }
      if (cols <= 0) {   // a narrow last tile has no slice for these warps
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
    }
    if (lane == 0) tma_store_done();
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
