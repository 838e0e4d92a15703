// Host side of the operators beside the block: q/k norm with rotation, gated scan, 8-bit projection.  Included by
// mate_api.cu (it uses that file's validation, trace and launch helpers).
#pragma once

namespace {

// What the kernels read and write in pairs of floats or one by one; rows of tensors start on 16 bytes (aligned16).
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// ------------------------------------------------------------------------------ q/k norm with rotation
mate_status check_qk(const mate_qk_config* c) {
  if (c == nullptr) return MATE_ERR_ARG;
  if (c->dtype != MATE_BF16 && c->dtype != MATE_F32) return MATE_ERR_ARG;
  if (c->pairing != 0 && c->pairing != 1) return MATE_ERR_ARG;
  if (!(c->eps > 0.f) || !std::isfinite(c->eps)) return MATE_ERR_ARG;
  if (c->B <= 0 || c->T <= 0 || c->H <= 0 || c->W <= 0 || c->hq <= 0 || c->hk <= 0 || c->hv < 0 || c->tp <= 0 ||
      c->rt < 0 || c->rh < 0 || c->rw < 0)
    return MATE_ERR_SHAPE;
  if (c->rt % 2 || c->rh % 2 || c->rw % 2 || (long long)c->rt + c->rh + c->rw > c->tp) return MATE_ERR_SHAPE;
  const int es = c->dtype == MATE_BF16 ? 2 : 4;
  if (c->tp > kQkMaxDim) return MATE_ERR_UNSUPPORTED;
  if (c->tp * es % 16) return MATE_ERR_SHAPE;
  if (((long long)c->hq + c->hk + c->hv) * c->tp >= (1LL << 31)) return MATE_ERR_SHAPE;
  // 64-bit products of three factors below 2^31 fit; a fourth is checked by division
  const long long hw = (long long)c->H * c->W;
  if (hw >= (1LL << 31) || hw * c->T >= (1LL << 31) || hw * c->T * c->B >= (1LL << 31)) return MATE_ERR_SHAPE;
  return MATE_OK;
}

// Row stride in elements, below 2^31: rows start on 16 bytes and hold `width` elements.
bool row_stride_ok(long long ld, long long width, int es) {
  return ld >= width && ld < (1LL << 31) && ld * es % 16 == 0;
}

mate_status fill_qk(const mate_qk_config* c, const void* x, long long ldx, const float* wq, const float* wk,
                    const float* tt, const float* th, const float* tw, QkParams* p) {
  const long long width = ((long long)c->hq + c->hk + c->hv) * c->tp;
  const int es = c->dtype == MATE_BF16 ? 2 : 4;
  if (x == nullptr || !aligned16(x) || !aligned8(wq) || !aligned8(wk) || !row_stride_ok(ldx, width, es))
    return MATE_ERR_ARG;
  if ((c->rt > 0 && tt == nullptr) || (c->rh > 0 && th == nullptr) || (c->rw > 0 && tw == nullptr) || !aligned8(tt) ||
      !aligned8(th) || !aligned8(tw))
    return MATE_ERR_ARG;
  p->x = x;
  p->ldx = ldx;
  p->wq = wq;
  p->wk = wk;
  p->tab_t = reinterpret_cast<const float2*>(tt);
  p->tab_h = reinterpret_cast<const float2*>(th);
  p->tab_w = reinterpret_cast<const float2*>(tw);
  p->rows = (long long)c->B * c->T * c->H * c->W;
  p->n = FastDiv(c->T * c->H * c->W);
  p->H = FastDiv(c->H);
  p->W = FastDiv(c->W);
  p->hq = c->hq;
  p->hk = c->hk;
  p->hv = c->hv;
  p->tp = c->tp;
  p->rt = c->rt;
  p->rh = c->rh;
  p->rw = c->rw;
  p->pairing = c->pairing;
  p->eps = c->eps;
  return MATE_OK;
}

// The kernel for a head's size and pairing: V channels per 16-byte unit, units of 32 lanes (fp32 heads of more than 128
// channels: two per lane), a power of two of lanes per head.
template <typename T_, int MODE, bool BWD>
void (*qk_kernel_of(int units))(QkParams) {
#define MATE_QK(NV, G) (BWD ? qk_norm_rope_bwd_kernel<T_, MODE, NV, G> : qk_norm_rope_kernel<T_, MODE, NV, G>)
  if constexpr (sizeof(T_) == 4)
    if (units > 32) return MATE_QK(2, 32);
  if (units > 16) return MATE_QK(1, 32);
  if (units > 8) return MATE_QK(1, 16);
  if (units > 4) return MATE_QK(1, 8);
  return MATE_QK(1, 4);
#undef MATE_QK
}

template <bool BWD>
mate_status launch_qk(int kid, const mate_qk_config* c, QkParams p, cudaStream_t st, int* blocks) {
  const int es = c->dtype == MATE_BF16 ? 2 : 4, V = 16 / es, units = c->tp / V;
  // halves whose axes are whole 8-byte units pair up inside a lane
  const int mode = c->pairing == 0 ? kQkAdjacent : (c->rt % V || c->rh % V || c->rw % V) ? kQkAny : kQkHalves;
  void (*kernel)(QkParams);
  if (es == 2)
    kernel = mode == kQkAdjacent ? qk_kernel_of<__nv_bfloat16, kQkAdjacent, BWD>(units)
                                 : mode == kQkHalves ? qk_kernel_of<__nv_bfloat16, kQkHalves, BWD>(units)
                                                     : qk_kernel_of<__nv_bfloat16, kQkAny, BWD>(units);
  else
    kernel = mode == kQkAdjacent ? qk_kernel_of<float, kQkAdjacent, BWD>(units)
                                 : mode == kQkHalves ? qk_kernel_of<float, kQkHalves, BWD>(units)
                                                     : qk_kernel_of<float, kQkAny, BWD>(units);
  // few rows: several warps share a row's heads
  const long long warps = 16LL * device_sms();
  const int per = 32 / std::min(32, units > 16 ? 32 : units > 8 ? 16 : units > 4 ? 8 : 4);
  const int iters = std::max(ceil_div(c->hq, per), ceil_div(c->hk, per));
  const int splits = static_cast<int>(std::max<long long>(1, std::min<long long>(iters, warps / p.rows)));
  p.splits = FastDiv(splits);
  // the backward pass with as many blocks as are resident, so that their weight gradients are few
  *blocks = static_cast<int>(std::min<long long>((p.rows * splits + kQkWarps - 1) / kQkWarps,
                                                 BWD ? std::min(kQkMaxParts, 2 * device_sms()) : 8 * device_sms()));
  trace_begin(kid, st);
  kernel<<<*blocks, kQkWarps * 32, 0, st>>>(p);
  MATE_LAUNCH_CHECK();
  return MATE_OK;
}

}  // namespace

extern "C" {

mate_status mate_rope_table(float* table, long long start, int count, int dims, double theta, mate_stream_t stream) {
  if (table == nullptr || !aligned8(table) || !(theta > 0.0) || !std::isfinite(theta)) return MATE_ERR_ARG;
  if (count <= 0 || dims <= 0 || dims % 2) return MATE_ERR_SHAPE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  t_launches = 0;
  const long long total = (long long)count * (dims / 2);
  trace_begin(MATE_K_ROPE_TABLE, st);
  rope_table_kernel<<<static_cast<int>(std::min<long long>((total + 255) / 256, 4096)), 256, 0, st>>>(
      reinterpret_cast<float2*>(table), static_cast<double>(start), count, dims / 2, theta);
  MATE_LAUNCH_CHECK();
  return MATE_OK;
}

mate_status mate_qk_norm_rope(const void* qkv, long long ldi, const float* wq, const float* wk, const float* tab_t,
                              const float* tab_h, const float* tab_w, void* out, long long ldo,
                              const mate_qk_config* cfg, mate_stream_t stream) {
  MATE_TRY(check_qk(cfg));
  QkParams p{};
  MATE_TRY(fill_qk(cfg, qkv, ldi, wq, wk, tab_t, tab_h, tab_w, &p));
  const int es = cfg->dtype == MATE_BF16 ? 2 : 4;
  if (out == nullptr || !aligned16(out) ||
      !row_stride_ok(ldo, ((long long)cfg->hq + cfg->hk + cfg->hv) * cfg->tp, es) || (out == qkv && ldo != ldi))
    return MATE_ERR_ARG;
  p.out = out;
  p.ldo = ldo;
  p.copy_v = cfg->hv > 0 && out != qkv;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  t_launches = 0;
  int blocks = 0;
  return launch_qk<false>(MATE_K_QK_NORM_ROPE, cfg, p, st, &blocks);
}

size_t mate_qk_norm_rope_backward_workspace_bytes(const mate_qk_config* cfg) {
  if (check_qk(cfg) != MATE_OK) return 0;
  return (size_t)kQkMaxParts * 2 * cfg->tp * sizeof(float);
}

mate_status mate_qk_norm_rope_backward(const void* qkv, long long ldi, const float* wq, const float* wk,
                                       const float* tab_t, const float* tab_h, const float* tab_w, const void* dout,
                                       long long ldg, void* dqkv, long long ldd, float* dwq, float* dwk,
                                       const mate_qk_config* cfg, void* ws, size_t ws_bytes, mate_stream_t stream) {
  MATE_TRY(check_qk(cfg));
  QkParams p{};
  MATE_TRY(fill_qk(cfg, qkv, ldi, wq, wk, tab_t, tab_h, tab_w, &p));
  const int es = cfg->dtype == MATE_BF16 ? 2 : 4;
  const long long width = ((long long)cfg->hq + cfg->hk + cfg->hv) * cfg->tp;
  if (dout == nullptr || dqkv == nullptr || ws == nullptr || !aligned16(dout) || !aligned16(dqkv) || !aligned16(ws) ||
      !row_stride_ok(ldg, width, es) || !row_stride_ok(ldd, width, es) || (dqkv == dout && ldd != ldg) ||
      (dqkv == qkv && ldd != ldi))
    return MATE_ERR_ARG;
  if (ws_bytes < mate_qk_norm_rope_backward_workspace_bytes(cfg)) return MATE_ERR_WORKSPACE;
  p.out = dqkv;
  p.ldo = ldd;
  p.dz = dout;
  p.ldz = ldg;
  p.part = static_cast<float*>(ws);
  p.copy_v = cfg->hv > 0 && dqkv != dout;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  t_launches = 0;
  int blocks = 0;
  MATE_TRY(launch_qk<true>(MATE_K_QK_NORM_ROPE_BWD, cfg, p, st, &blocks));
  if (dwq != nullptr || dwk != nullptr) {
    trace_begin(MATE_K_QK_WEIGHT_GRAD, st);
    sum_parts_kernel<<<ceil_div(2 * cfg->tp, 32), 1024, 0, st>>>(p.part, blocks, 2 * cfg->tp, dwq, cfg->tp, dwk);
    MATE_LAUNCH_CHECK();
  }
  return MATE_OK;
}

}  // extern "C"

// ------------------------------------------------------------------------------ gated scan
namespace {

// Rows per chunk: long chunks carry little, but there have to be threads enough (four channels of a chunk each) to fill
// the SMs.  The number of threads is fixed, not asked of the device: the workspace's size goes by cfg alone and has to be the
// same wherever the call runs, and so do the results, which a chunk's border rounds.
constexpr long long kGsFillThreads = 1024LL * 148;
int gated_chunk(const mate_gated_scan_config* c) {
  const long long n = (long long)c->T * c->H * c->W, cols = (long long)c->B * (c->D / 4);
  if (n <= kGsOneChunk) return static_cast<int>(n);
  int r = kGsMaxChunk;
  while (r > 16 && (n + r - 1) / r * cols < kGsFillThreads) r /= 2;
  return r;
}

int gated_chunks(const mate_gated_scan_config* c) { return ceil_div((long long)c->T * c->H * c->W, gated_chunk(c)); }

mate_status check_gated(const mate_gated_scan_config* c) {
  if (c == nullptr) return MATE_ERR_ARG;
  if (c->dtype != MATE_BF16 && c->dtype != MATE_F32) return MATE_ERR_ARG;
  if (c->order < 0 || c->order > 3 || (c->reverse != 0 && c->reverse != 1)) return MATE_ERR_ARG;
  if (c->B <= 0 || c->T <= 0 || c->H <= 0 || c->W <= 0 || c->D <= 0) return MATE_ERR_SHAPE;
  if (c->D % (c->dtype == MATE_BF16 ? 8 : 4)) return MATE_ERR_SHAPE;
  const long long hw = (long long)c->H * c->W;
  if (hw >= (1LL << 31) || hw * c->T >= (1LL << 31) || hw * c->T * c->B >= (1LL << 31)) return MATE_ERR_SHAPE;
  // threads of two channels of a chunk, and columns of all samples, are counted in 31 bits
  if ((long long)c->B * c->D >= (1LL << 31) || (long long)gated_chunks(c) * c->B >= (1LL << 31) / (c->D / 2))
    return MATE_ERR_SHAPE;
  return MATE_OK;
}

// The grid rows along scan order `order` (fastest axis first), `reverse`: from the last position.
GsOrder gated_order(const mate_gated_scan_config* c, int reverse) {
  const int H = c->H, W = c->W, T = c->T, n = T * H * W;
  int dim[3], step[3];
  switch (c->order) {
    case 0: dim[0] = n, dim[1] = dim[2] = 1, step[0] = 1, step[1] = step[2] = 0; break;
    case 1: dim[0] = H, dim[1] = W, dim[2] = T, step[0] = W, step[1] = 1, step[2] = H * W; break;
    case 2: dim[0] = T, dim[1] = W, dim[2] = H, step[0] = H * W, step[1] = 1, step[2] = W; break;
    default: dim[0] = T, dim[1] = H, dim[2] = W, step[0] = H * W, step[1] = W, step[2] = 1; break;
  }
  GsOrder o;
  o.base = 0;
  if (reverse)
    for (int i = 0; i < 3; ++i) {
      o.base += (dim[i] - 1) * step[i];
      step[i] = -step[i];
    }
  o.n0 = FastDiv(dim[0]);
  o.n1 = FastDiv(dim[1]);
  o.s0 = step[0];
  o.d1 = step[1] - dim[0] * step[0];
  o.d2 = step[2] - dim[1] * step[1];
  return o;
}

mate_status fill_gated(const mate_gated_scan_config* c, const void* x, long long ldx, const void* g, long long ldg,
                       const float* bias, GatedScanParams* p) {
  const int es = c->dtype == MATE_BF16 ? 2 : 4;
  if (x == nullptr || g == nullptr || !aligned16(x) || !aligned16(g) || !aligned8(bias) ||
      !row_stride_ok(ldx, c->D, es) || !row_stride_ok(ldg, c->D, es))
    return MATE_ERR_ARG;
  p->x = x;
  p->g = g;
  p->ldx = static_cast<unsigned>(ldx);
  p->ldg = static_cast<unsigned>(ldg);
  p->bias = bias;
  p->order = gated_order(c, c->reverse);
  p->back = gated_order(c, !c->reverse);
  p->B = FastDiv(c->B);
  p->D = c->D;
  p->n = c->T * c->H * c->W;
  p->chunk = gated_chunk(c);
  p->chunks = gated_chunks(c);
  p->states_per = ceil_div(p->n, kGsState);
  return MATE_OK;
}

struct GatedScanScratch {
  float2* pair;
  float* carry;
  float* dbias_part;
  size_t bytes;
};

// A sequence of one chunk joins nothing.
GatedScanScratch carve_gated(const mate_gated_scan_config* c, void* ws, bool backward) {
  GatedScanScratch s{};
  Carver cv{static_cast<char*>(ws)};
  const size_t chunks = gated_chunks(c), cols = (size_t)c->B * c->D;
  if (chunks > 1) {
    s.pair = cv.take<float2>(chunks * cols);
    s.carry = cv.take<float>(chunks * cols);
  }
  if (backward) s.dbias_part = cv.take<float>(chunks * cols);
  s.bytes = cv.off;
  return s;
}

// Grid of a kernel whose threads take 2 np channels of a chunk.
int gated_blocks(GatedScanParams* p, int np, int threads) {
  p->per = FastDiv(p->D / (2 * np));
  p->threads = static_cast<unsigned>(p->chunks) * p->B.d * p->per.d;
  return static_cast<int>((p->threads + threads - 1u) / threads);
}

mate_status launch_carry(const GatedScanParams& p, const float* start, int back, cudaStream_t st) {
  const int cols = static_cast<int>(p.B.d) * p.D;
  trace_begin(MATE_K_GATED_SCAN_CARRY, st);
  if (p.chunks <= 8 * kGsCarryHeld)
    gated_carry_kernel<32, 8><<<ceil_div(cols, 32), 256, 0, st>>>(p.pair, start, p.carry, p.chunks, cols, back);
  else if (p.chunks <= 32 * kGsCarryHeld)
    gated_carry_kernel<16, 32><<<ceil_div(cols, 16), 512, 0, st>>>(p.pair, start, p.carry, p.chunks, cols, back);
  else
    gated_carry_kernel<8, 64><<<ceil_div(cols, 8), 512, 0, st>>>(p.pair, start, p.carry, p.chunks, cols, back);
  MATE_LAUNCH_CHECK();
  return MATE_OK;
}

}  // namespace

extern "C" {

size_t mate_gated_scan_workspace_bytes(const mate_gated_scan_config* cfg) {
  if (check_gated(cfg) != MATE_OK) return 0;
  return carve_gated(cfg, nullptr, false).bytes;
}

size_t mate_gated_scan_states_bytes(const mate_gated_scan_config* cfg) {
  if (check_gated(cfg) != MATE_OK) return 0;
  return (size_t)cfg->B * ceil_div((long long)cfg->T * cfg->H * cfg->W, kGsState) * cfg->D * sizeof(float);
}

mate_status mate_gated_scan(const void* x, long long ldx, const void* g, long long ldg, const float* bias,
                            const float* h0, void* y, long long ldy, float* h_last, float* states,
                            const mate_gated_scan_config* cfg, void* ws, size_t ws_bytes, mate_stream_t stream) {
  MATE_TRY(check_gated(cfg));
  GatedScanParams p{};
  MATE_TRY(fill_gated(cfg, x, ldx, g, ldg, bias, &p));
  const bool bf = cfg->dtype == MATE_BF16;
  const size_t need = mate_gated_scan_workspace_bytes(cfg);
  if (y == nullptr || y == x || y == g || !aligned16(y) || !row_stride_ok(ldy, cfg->D, bf ? 2 : 4) || !aligned8(h0) ||
      !aligned8(h_last) || !aligned8(states) || !aligned16(ws) || (ws == nullptr && need > 0))
    return MATE_ERR_ARG;
  if (ws_bytes < need) return MATE_ERR_WORKSPACE;
  const GatedScanScratch s = carve_gated(cfg, ws, false);
  p.h0 = h0;
  p.y = y;
  p.ldy = static_cast<unsigned>(ldy);
  p.h_last = h_last;
  p.states = states;
  p.pair = s.pair;
  p.carry = s.carry;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  t_launches = 0;
  const int blocks = gated_blocks(&p, 2, kGsThreads);
  if (p.chunks > 1) {
    trace_begin(MATE_K_GATED_SCAN_PAIRS, st);
    if (bf) gated_scan_kernel<__nv_bfloat16, false><<<blocks, kGsThreads, 0, st>>>(p);
    else gated_scan_kernel<float, false><<<blocks, kGsThreads, 0, st>>>(p);
    MATE_LAUNCH_CHECK();
    MATE_TRY(launch_carry(p, h0, 0, st));
  }
  trace_begin(MATE_K_GATED_SCAN, st);
  if (bf) gated_scan_kernel<__nv_bfloat16, true><<<blocks, kGsThreads, 0, st>>>(p);
  else gated_scan_kernel<float, true><<<blocks, kGsThreads, 0, st>>>(p);
  MATE_LAUNCH_CHECK();
  return MATE_OK;
}

size_t mate_gated_scan_backward_workspace_bytes(const mate_gated_scan_config* cfg) {
  if (check_gated(cfg) != MATE_OK) return 0;
  return carve_gated(cfg, nullptr, true).bytes;
}

mate_status mate_gated_scan_backward(const void* x, long long ldx, const void* g, long long ldg, const float* bias,
                                     const float* states, const void* dy, long long lddy, const float* dh_last,
                                     void* dx, long long lddx, void* dg, long long lddg, float* dbias, float* dh0,
                                     const mate_gated_scan_config* cfg, void* ws, size_t ws_bytes,
                                     mate_stream_t stream) {
  MATE_TRY(check_gated(cfg));
  GatedScanParams p{};
  MATE_TRY(fill_gated(cfg, x, ldx, g, ldg, bias, &p));
  const bool bf = cfg->dtype == MATE_BF16;
  const int es = bf ? 2 : 4;
  if (states == nullptr || dy == nullptr || dx == nullptr || dg == nullptr || ws == nullptr || !aligned8(states) ||
      !aligned16(dy) || !aligned16(dx) || !aligned16(dg) || !aligned8(dh_last) || !aligned8(dbias) ||
      !aligned8(dh0) || !aligned16(ws) || !row_stride_ok(lddy, cfg->D, es) || !row_stride_ok(lddx, cfg->D, es) ||
      !row_stride_ok(lddg, cfg->D, es))
    return MATE_ERR_ARG;
  for (const void* in : {x, g, dy})
    if (dx == in || dg == in) return MATE_ERR_ARG;
  if (dx == dg) return MATE_ERR_ARG;
  if (ws_bytes < mate_gated_scan_backward_workspace_bytes(cfg)) return MATE_ERR_WORKSPACE;
  const GatedScanScratch s = carve_gated(cfg, ws, true);
  p.states = const_cast<float*>(states);
  p.dy = dy;
  p.lddy = static_cast<unsigned>(lddy);
  p.dh_last = dh_last;
  p.dx = dx;
  p.lddx = static_cast<unsigned>(lddx);
  p.dg = dg;
  p.lddg = static_cast<unsigned>(lddg);
  p.dbias_part = dbias != nullptr ? s.dbias_part : nullptr;
  p.dh0 = dh0;
  p.pair = s.pair;
  p.carry = s.carry;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  t_launches = 0;
  if (p.chunks > 1) {
    const int blocks = gated_blocks(&p, 2, kGsThreads);
    trace_begin(MATE_K_GATED_SCAN_PAIRS, st);
    if (bf) gated_adjoint_kernel<__nv_bfloat16><<<blocks, kGsThreads, 0, st>>>(p);
    else gated_adjoint_kernel<float><<<blocks, kGsThreads, 0, st>>>(p);
    MATE_LAUNCH_CHECK();
    MATE_TRY(launch_carry(p, dh_last, 1, st));
  }
  const int blocks = gated_blocks(&p, 1, kGsBwdThreads);
  trace_begin(MATE_K_GATED_SCAN_BWD, st);
  if (bf) gated_scan_bwd_kernel<__nv_bfloat16><<<blocks, kGsBwdThreads, 0, st>>>(p);
  else gated_scan_bwd_kernel<float><<<blocks, kGsBwdThreads, 0, st>>>(p);
  MATE_LAUNCH_CHECK();
  if (dbias != nullptr) {
    trace_begin(MATE_K_GATED_SCAN_BIAS, st);
    sum_parts_kernel<<<ceil_div(cfg->D, 32), 1024, 0, st>>>(s.dbias_part, cfg->B * p.chunks, cfg->D, dbias, cfg->D, nullptr);
    MATE_LAUNCH_CHECK();
  }
  return MATE_OK;
}

}  // extern "C"

// ------------------------------------------------------------------------------ 8-bit projection
namespace {

// Rows and columns are counted in 32 bits, and the kernels step past the last one by up to a grid's share of rows (8 blocks
// of 8 rows on every SM) or a tile's of columns before they compare: the sizes stay that far below 2^31.
constexpr long long kI8MaxSize = (1LL << 31) - (1LL << 14);

// 2D matrix of bytes [rows, cols], row stride ld (a multiple of 16); box = box_rows x 128 columns, 128B swizzle.
// Columns and rows behind the matrix read zeros.
bool make_tmap_s8(CUtensorMap* m, const void* ptr, long long rows, long long cols, long long ld, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output matrix [rows, cols], box = 32 x 32; 64-byte swizzle for 2-byte elements, 128-byte for 4-byte ones.
bool make_tmap_out(CUtensorMap* m, void* ptr, long long rows, int cols, long long ld, int es) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, ptr, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, es == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A warp per row where there are rows enough to fill the SMs and a warp can hold one, else a block per row (bf16,
// K = 2048: 512 rows 2.6 us by warps, 2.2 by blocks; 1184 rows 2.9 and 3.4; 4736 rows 5.4 and 8.8).
template <typename T_, int G>
auto quantize_kernel_of(int vectors) -> void (*)(const T_*, long long, int, int, int8_t*, long long, float*) {
  if (vectors <= G) return quantize_rows_kernel<T_, G, 1>;
  if (vectors <= 2 * G) return quantize_rows_kernel<T_, G, 2>;
  if (vectors <= 4 * G) return quantize_rows_kernel<T_, G, 4>;
  if (G > 32 && vectors > 8 * G) return quantize_rows_kernel<T_, 256, 0>;
  return quantize_rows_kernel<T_, G, 8>;
}

template <typename T_>
void launch_quantize(const T_* x, long long ldx, int M, int K, void* q, long long ldq, float* scale, cudaStream_t st) {
  const int sms = device_sms(), vectors = K / (16 / static_cast<int>(sizeof(T_)));
  const bool warps = M >= 6 * sms && vectors <= 8 * 32;
  auto kernel = warps ? quantize_kernel_of<T_, 32>(vectors) : quantize_kernel_of<T_, 256>(vectors);
  const int blocks = std::min(warps ? ceil_div(M, 8) : M, 8 * sms);
  kernel<<<blocks, 256, 0, st>>>(x, ldx, M, K, static_cast<int8_t*>(q), ldq, scale);
}

template <typename T_>
void launch_int8_few(const int8_t* A, long long lda, const float* a_scale, int M, int K, const int8_t* W, long long ldw,
                     const float* w_scale, int N, const float* bias, void* C, long long ldc, cudaStream_t st) {
  T_* c = static_cast<T_*>(C);
  const int blocks = ceil_div(N, 4 * kFewCols);
  auto kernel = M == 1   ? gemm_int8_few_kernel<T_, 1>
                : M == 2 ? gemm_int8_few_kernel<T_, 2> : gemm_int8_few_kernel<T_, kFewRows>;
  kernel<<<blocks, 128, 0, st>>>(A, lda, a_scale, M, K, W, ldw, w_scale, N, bias, c, ldc);
}

}  // namespace

extern "C" {

mate_status mate_quantize_rows(const void* x, long long ldx, long long M, int K, mate_dtype dtype, void* q,
                               long long ldq, float* scale, mate_stream_t stream) {
  if (dtype != MATE_BF16 && dtype != MATE_F32) return MATE_ERR_ARG;
  const int es = dtype == MATE_BF16 ? 2 : 4;
  if (x == nullptr || q == nullptr || scale == nullptr || M < 0 || K <= 0 || M > kI8MaxSize || K > kI8MaxSize)
    return MATE_ERR_ARG;
  if (!aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scale) & 3u) || !row_stride_ok(ldx, K, es) ||
      !row_stride_ok(ldq, K, 1))
    return MATE_ERR_ARG;
  t_launches = 0;
  if (M == 0) return MATE_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  trace_begin(MATE_K_QUANTIZE_ROWS, st);
  const int m = static_cast<int>(M);
  if (dtype == MATE_BF16) launch_quantize(static_cast<const __nv_bfloat16*>(x), ldx, m, K, q, ldq, scale, st);
  else launch_quantize(static_cast<const float*>(x), ldx, m, K, q, ldq, scale, st);
  MATE_LAUNCH_CHECK();
  return MATE_OK;
}

mate_status mate_project_int8(const void* A, long long lda, const float* a_scale, long long M, int K, const void* Wt,
                              long long ldw, const float* w_scale, int N, const float* bias, void* C, long long ldc,
                              mate_dtype out_dtype, mate_stream_t stream) {
  if (out_dtype != MATE_BF16 && out_dtype != MATE_F32) return MATE_ERR_ARG;
  if (A == nullptr || a_scale == nullptr || Wt == nullptr || w_scale == nullptr || C == nullptr || M < 0 || K <= 0 ||
      N <= 0 || M > kI8MaxSize || N > kI8MaxSize)
    return MATE_ERR_ARG;
  if (!aligned16(A) || !aligned16(Wt) || !aligned8(C) || !aligned8(w_scale) || !aligned8(bias) ||
      (reinterpret_cast<uintptr_t>(a_scale) & 3u) || !row_stride_ok(lda, K, 1) || !row_stride_ok(ldw, K, 1) || ldc < N ||
      ldc >= (1LL << 31))
    return MATE_ERR_ARG;
  if (K >= 131072) return MATE_ERR_UNSUPPORTED;
  t_launches = 0;
  if (M == 0) return MATE_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (M <= kFewRows) {
    const int8_t *a = static_cast<const int8_t*>(A), *w = static_cast<const int8_t*>(Wt);
    trace_begin(MATE_K_PROJECT_INT8, st);
    if (out_dtype == MATE_BF16)
      launch_int8_few<__nv_bfloat16>(a, lda, a_scale, static_cast<int>(M), K, w, ldw, w_scale, N, bias, C, ldc, st);
    else
      launch_int8_few<float>(a, lda, a_scale, static_cast<int>(M), K, w, ldw, w_scale, N, bias, C, ldc, st);
    MATE_LAUNCH_CHECK();
    return MATE_OK;
  }
  Int8GemmParams p;
  p.M = static_cast<int>(M);
  p.N = N;
  p.K = K;
  // Tile width: 256, which feeds the MMAs best, unless there are fewer such tiles than pairs of SMs; then the one whose
  // rounds over the pairs are the shortest (a tile costs its columns of W and a start).  16 x 2048 x 12288: 12.0 us at 256
  // columns, 16.5 at 128, 21 at 64; 16 x 1024 x 4096: 8.7, 7.3 and 6.9.
  const int pairs_all = device_sms() / 2;
  p.bn = 256;
  if ((long long)ceil_div(M, 256) * ceil_div(N, 256) < pairs_all) {
    long long best = 1LL << 62;
    for (int bn = 256; bn >= 32; bn /= 2) {
      const long long tiles = (long long)ceil_div(M, 256) * ceil_div(N, bn);
      const long long cost = (long long)ceil_div(tiles, pairs_all) * (bn + kI8TileStart);
      if (cost < best) {
        best = cost;
        p.bn = bn;
      }
    }
  }
  p.num_n_tiles = ceil_div(N, p.bn);
  const long long tiles = (long long)ceil_div(M, 256) * p.num_n_tiles;
  if (tiles >= (1LL << 31)) return MATE_ERR_SHAPE;
  p.num_tiles = static_cast<int>(tiles);
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.bias = bias;
  p.C = C;
  p.ldc = ldc;
  p.vec = aligned16(C) && ldc * (out_dtype == MATE_BF16 ? 2 : 4) % 16 == 0;
  // Keep W in shared memory where that is the shorter way: its tiles take 1 / kI8KeepGain of the others' time, but the
  // pairs share out whole column tiles.  65536 x 1024 x 4368 (64 tiles a pair against 63): 250 us against 263;
  // 16384 x 1024 x 4096 (16 against 14): 68 against 60.  fp32 output is staged in twice the space, and stops gaining where
  // W leaves fewer than five stages for A.  65536 rows, fp32: K = 512, N = 4368 213 us kept, 220 streamed; K = 768, N = 2048
  // 119 and 119; K = 896, N = 2048 145 and 133; K = 1024, N = 4368 346 and 309.
  constexpr double kI8KeepGain = 1.1;
  const int mblocks = ceil_div(M, 256);
  int pairs = std::min(p.num_tiles, pairs_all);
  p.slots = std::min(p.num_n_tiles, pairs_all);
  p.groups = std::min(pairs_all / p.slots, mblocks);
  const long long kept_tiles = (long long)ceil_div(p.num_n_tiles, p.slots) * ceil_div(mblocks, p.groups);
  const int es = out_dtype == MATE_BF16 ? 2 : 4;
  const bool keep = K <= (es == 2 ? kI8KeepK : kI8KeepKF32) && p.bn == 256 && kept_tiles < kI8KeepGain * ceil_div(p.num_tiles, pairs);
  if (keep) pairs = p.slots * p.groups;
  const uint32_t sb = int8_stage_bytes(p.bn, keep);
  const uint32_t fixed = 1024 + int8_kept_bytes(p.bn, K, keep) + int8_out_bytes(es) + kI8Behind;
  p.stages = std::min<int>(8, static_cast<int>((kSmemLimit - fixed) / sb));
  Int8Maps maps;
  if (!make_tmap_s8(&maps.a, A, M, K, lda, 128) || !make_tmap_s8(&maps.w, Wt, N, K, ldw, p.bn / 2)) return MATE_ERR_CUDA;
  if (p.vec) {
    if (!make_tmap_out(&maps.c, C, M, N, ldc, es)) return MATE_ERR_CUDA;
  } else {
    maps.c = maps.a;   // never used
  }
  const size_t smem = fixed + (size_t)p.stages * sb;
  auto kernel = es == 2 ? (keep ? gemm_int8_pair_kernel<__nv_bfloat16, true> : gemm_int8_pair_kernel<__nv_bfloat16, false>)
                        : (keep ? gemm_int8_pair_kernel<float, true> : gemm_int8_pair_kernel<float, false>);
  if (!set_smem(kernel, smem)) return MATE_ERR_CUDA;
  trace_begin(MATE_K_PROJECT_INT8, st);
  kernel<<<2 * pairs, kI8Threads, smem, st>>>(maps, p);
  MATE_LAUNCH_CHECK();
  return MATE_OK;
}

}  // extern "C"
