// C ABI of the operators around a decode step (include/moe.h): the norm before the layer, MXFP4
// linears, and the layer for a few tokens.  Included by api.cu, whose helpers it uses.
#pragma once

namespace {

// The weights' and the token rows' maps of few_kernel: tile-major weights as the grouped GEMM reads them,
// token rows in boxes of 16.
bool make_few_maps(CUtensorMap* mW, CUtensorMap* mX, const void* w, uint64_t tiles, const void* x, uint64_t rows, int K) {
  return make_map(mW, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, w, 128, tiles * 256, 64, 128, 256) &&
         make_map(mX, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, K, rows, K, 128, kFewRows);
}

// Pipeline stages that fit next to few_kernel's tables; it wants three at least.
int few_stages(int mode, int T, int k, int k_tiles) {
  const long long fixed = few_smem(mode, T, k, k_tiles, 0).total;
  return (int)std::min<long long>(kFewMaxStages, (kFewSmemMax - fixed) / (kFewStage + kFewSF));
}
constexpr int kFewMinStages = 3;

// Launch few_kernel with as many pipeline stages as fit.
template <int MODE, int ACT>
cudaError_t launch_few(FewArgs a, const CUtensorMap& tW, const CUtensorMap& tX, const CUtensorMap& tSW, const CUtensorMap& tSX,
                       int grid, cudaStream_t s) {
  auto kern = few_kernel<MODE, ACT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_attr(kern, kFewSmemMax, done);
  if (e != cudaSuccess) return e;
  a.stages = few_stages(MODE, a.T, a.k, a.k_tiles);
  if (a.stages < kFewMinStages) return cudaErrorInvalidValue;   // the callers check before any launch
  a.by_m = fast_div(a.m_tiles);
  a.by_k = fast_div(a.k_tiles);
  a.by_ss = fast_div(std::max(2 * a.sh_steps, 1));
  a.by_grid = fast_div(grid);
  return launch_k(kern, grid, kFewThreads, few_smem(MODE, a.T, a.k, a.k_tiles, a.stages).total, s, a, tW, tX, tSW, tSX);
}

template <int NB>
cudaError_t launch_linear(const LinearArgs& a, const CUtensorMap& tW, const CUtensorMap& tX, cudaStream_t s) {
  auto kern = linear_kernel<NB>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem_attr(kern, LinearCfg<NB>::SMEM, done);
  if (e != cudaSuccess) return e;
  e = launch_k(kern, a.ctas, kLinearThreads, LinearCfg<NB>::SMEM, s, a, tW, tX);
  if (e == cudaSuccess && a.unit < a.k_tiles)
    e = launch_k(linear_sum_kernel, dim3(a.n_tiles * a.m_tiles, a.n_per / 4), 256, 0, s, a);
  return e;
}

// The norm's variants.  A thread holds V vectors of 8 elements: one where a row fits 1024 threads so,
// else 2 or 4.  The streaming kernel pays where there are rows for more than one turn and a CTA per row
// has too few loads in flight.  With a bf16 residual that is where only two such CTAs fit an SM: 8192 x
// 7168 85.6 us against 96.4, 400 x 7168 7.72 against 7.77; but 8192 x 4096 52.2 against 49.6.  Without
// one, at half the loads, also narrower: 8192 x 7168 57.5 against 80.7, 8192 x 4096 32.2 against 39.3,
// 8192 x 2048 (left as it is) 18.9 against 19.4.
constexpr int kNormStreamVecs = 512, kNormStreamVecsPlain = 256;
template <int RES, int V>
cudaError_t launch_norm_rows(const NormArgs& a, cudaStream_t s) {
  const int nvec = a.cols / 8, team = ((nvec + V - 1) / V + 31) / 32 * 32, per_cta = std::max(1, 128 / team);
  return launch_k(add_rmsnorm_mxfp8_kernel<RES, V>, (unsigned)((a.rows + per_cta - 1) / per_cta), dim3(team, per_cta), 0, s, a);
}
template <int RES>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  const int nvec = a.cols / 8;
  if constexpr (RES != NORM_RES_F32) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return cudaErrorInvalidDevice;
    constexpr int V = kNormStreamVecsPerThread;
    const int team = ((nvec + V - 1) / V + 31) / 32 * 32, grid = sms * std::max(1, 1152 / team);   // as many as fit (56 registers a thread)
    if (nvec > (RES == NORM_RES_BF16 ? kNormStreamVecs : kNormStreamVecsPlain) && nvec <= 1024 * V && a.rows > grid) {
      auto kern = add_rmsnorm_mxfp8_stream_kernel<RES>;
      static std::atomic<uint64_t> done{0};
      const cudaError_t e = ensure_smem_attr(kern, kNormDepth * V * 32 * 1024, done);
      if (e != cudaSuccess) return e;
      return launch_k(kern, grid, team, kNormDepth * V * (RES == NORM_RES_BF16 ? 32 : 16) * team, s, a);
    }
  }
  if (nvec > 2048) return launch_norm_rows<RES, 4>(a, s);
  if (nvec > 1024) return launch_norm_rows<RES, 2>(a, s);
  return launch_norm_rows<RES, 1>(a, s);
}

}  // namespace

struct moe_linear_s {
  int T_max, N, K;
  int num_sms = 148;
  char* ws = nullptr;
  size_t o_status, o_cnt, o_part, total;
  int grid() const { return std::min(num_sms, kFewMaxCtas); }
  template <class P>
  P* at(size_t off) const { return (P*)(ws + off); }
};
// linear_kernel's tiles: up to 64 token rows with five pipeline stages, or up to 176 (the widest whose
// accumulators, with four stages' scales, fit the tensor memory and whose stages fit shared memory).
constexpr int kLinearSmall = 64, kLinearWide = 176;

// Token rows per tile (a multiple of 16) and whether tiles stay whole, by the time each choice takes, in
// ns, for every number of rows:
//   a step of n rows takes 255 + 0.77 n (n <= 64) or 190 + 2.1 n: up to 64 rows the issue and the weights,
//   above them the shared memory's fill rate;
//   whole tiles cost the last wave's idle SMs;
//   exchanging partials takes 2500 + 55 n, and 0.8 for each CTA of the kernel that adds them, four token
//   rows of a tile each (without it 2700 rows of 7168 x 7168 are split, 159 us instead of 122 whole, and
//   1024 rows of 28672 x 7168, 233 instead of 197).
// Fitted to ten shapes from 256 x 7168 to 28672 x 7168 with 17 to 8192 rows, every height and both forms
// timed: the choice takes 1.1% more than the best one on average.  300 rows of 7168 x 7168: five whole
// tiles of 64 rows by 28 take 20.9 us, 64 rows: one tile split 13.4, two whole ones 20.2.
struct LinearPick { int n_per, unit; };
LinearPick pick_linear_tiles(int T, int m_tiles, int k_tiles, int grid) {
  LinearPick best = {kLinearWide, k_tiles};
  double best_ns = 1e30;
  for (int n = 16; n <= kLinearWide; n += 16) {
    const long long tiles = (long long)((T + n - 1) / n) * m_tiles, steps = tiles * k_tiles;
    if (steps > 0x7fffffffll) continue;   // the kernel counts steps in 32 bits
    const double step = n <= kLinearSmall ? 255.0 + 0.77 * n : 190.0 + 2.1 * n;
    const double whole = (double)((tiles + grid - 1) / grid) * k_tiles * step;
    const long long ctas = std::max(std::min(steps / 4, (long long)grid), 1ll);
    const double split = (double)((steps + ctas - 1) / ctas) * step + 2500.0 + 55.0 * n + 0.8 * (double)(tiles * (n / 4));
    if (whole < best_ns) { best_ns = whole; best = {n, k_tiles}; }
    if (k_tiles > 1 && split < best_ns) { best_ns = split; best = {n, 1}; }
    if (n >= T) break;
  }
  return best;
}
// Whether a call with T rows is a stream of the weights (few.cuh).
bool linear_streams(int T, int k_tiles) { return T <= kFewRows && few_stages(FEW_LINEAR, T, 0, k_tiles) >= kFewMinStages; }

extern "C" {

moe_status_t moe_add_rmsnorm_mxfp8(const void* x, const void* residual, moe_type_t residual_type, const float* gamma,
                                   float eps, int rows, int cols, void* residual_out, void* xn, uint8_t* q,
                                   uint8_t* scale, void* stream) {
  if (rows < 0 || cols <= 0 || !(eps > 0.0f) || (residual_type != MOE_TYPE_BF16 && residual_type != MOE_TYPE_F32))
    return MOE_ERR_INVALID_ARG;
  if (cols % 32 || cols > kNormMaxCols) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if ((residual_out && !residual) || (q != nullptr) != (scale != nullptr) || !(residual_out || xn || q))
    return MOE_ERR_INVALID_ARG;
  if (!x || !gamma) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(residual_out, 16) || !aligned(xn, 16) ||
      !aligned(q, 16))
    return MOE_ERR_ALIGNMENT;
  NormArgs a{(const uint16_t*)x, residual, gamma, eps, rows, cols, residual_out, (uint16_t*)xn, q, scale};
  const int res = !residual ? NORM_RES_NONE : residual_type == MOE_TYPE_BF16 ? NORM_RES_BF16 : NORM_RES_F32;
  cudaError_t e;
  switch (res) {
    case NORM_RES_NONE: e = launch_norm<NORM_RES_NONE>(a, S(stream)); break;
    case NORM_RES_BF16: e = launch_norm<NORM_RES_BF16>(a, S(stream)); break;
    default: e = launch_norm<NORM_RES_F32>(a, S(stream)); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// ---------------------------------------------------------------- MXFP4 linear
moe_status_t moe_linear_create(int T_max, int N, int K, moe_linear_t* out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (T_max < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  const long long m_tiles = ((long long)N + 255) / 256;
  // tensor-map coordinates are 32-bit: tile rows of the weights, and token rows
  if (K % 128 || K > (1 << 22) || m_tiles * (K / 128) * 256 > (1ll << 30) || T_max > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  moe_linear_s* p = new moe_linear_s();
  p->T_max = T_max; p->N = N; p->K = K;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && sms > 0)
    p->num_sms = sms;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t r = o; o = up(o + bytes, 1024); return r; };
  p->o_status = take(256);
  p->o_cnt = take((size_t)kFewMaxCtas * 4);
  // fp32 partials of two ragged tiles per CTA
  p->o_part = take((size_t)2 * p->grid() * std::min(std::max((T_max + 15) / 16 * 16, 16), kLinearWide) * 256 * 4);
  p->total = o;
  *out = p;
  return MOE_OK;
}

moe_status_t moe_linear_workspace_bytes(moe_linear_t p, size_t* bytes) {
  if (!p || !bytes) return MOE_ERR_INVALID_ARG;
  *bytes = p->total;
  return MOE_OK;
}

moe_status_t moe_linear_set_workspace(moe_linear_t p, void* dev_ptr, size_t bytes) {
  if (!p || !dev_ptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(dev_ptr, 256)) return MOE_ERR_ALIGNMENT;
  if (bytes < p->total) return MOE_ERR_INVALID_ARG;
  p->ws = (char*)dev_ptr;
  // the status word and the tile counters
  if (cudaMemset(p->ws, 0, p->o_part) != cudaSuccess || cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status_t moe_linear_check(moe_linear_t p, void* stream, unsigned int* bits) {
  if (!p) return MOE_ERR_INVALID_ARG;
  if (!p->ws) return MOE_ERR_NOT_INITIALIZED;
  return take_status(p->at<unsigned int>(p->o_status), p->at<unsigned int>(p->o_cnt), S(stream), bits);
}

moe_status_t moe_linear_tiling(moe_linear_t p, int T, int* rows, int* split) {
  if (!p || T < 0 || !rows || !split) return MOE_ERR_INVALID_ARG;
  if (T > p->T_max) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int k_tiles = p->K / 128;
  *rows = *split = 0;
  if (T == 0 || linear_streams(T, k_tiles)) return MOE_OK;
  const LinearPick pick = pick_linear_tiles(T, (p->N + 255) / 256, k_tiles, p->grid());
  *rows = pick.n_per;
  *split = pick.unit < k_tiles;
  return MOE_OK;
}

moe_status_t moe_linear_destroy(moe_linear_t p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  delete p;
  return MOE_OK;
}

moe_status_t moe_linear_bytes(int N, int K, size_t* w, size_t* s) {
  if (N <= 0 || K <= 0 || !w || !s) return MOE_ERR_INVALID_ARG;
  if (K % 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  const size_t tiles = ((size_t)N + 255) / 256 * (K / 128);
  *w = tiles * kFewTile;
  *s = tiles * 1024;
  return MOE_OK;
}

moe_status_t moe_pack_linear_mxfp4(int N, int K, const float* src, const moe_matrix_mxfp4* dst, void* stream) {
  size_t nw = 0, ns = 0;
  if (!src || !dst || !dst->w || !dst->s) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = moe_linear_bytes(N, K, &nw, &ns);
  if (st != MOE_OK) return st;
  if (!aligned(src, 16) || !aligned(dst->w, 256) || !aligned(dst->s, 16)) return MOE_ERR_ALIGNMENT;
  const long long n = (long long)N * (K / 32);
  if ((n + 255) / 256 > 0x7fffffffll) return MOE_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = S(stream);
  // rows past N in the last 256-row tile are zeros
  if (N % 256 && (cudaMemsetAsync(dst->w, 0, nw, s) != cudaSuccess || cudaMemsetAsync(dst->s, 0, ns, s) != cudaSuccess))
    return MOE_ERR_CUDA;
  pack_mxfp4_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(src, nullptr, N, K, 0, (uint8_t*)dst->w, (uint8_t*)dst->s);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_linear_mxfp4(moe_linear_t p, const uint8_t* q, const uint8_t* scale, int T, const moe_matrix_mxfp4* W,
                              void* y, moe_type_t y_type, void* stream) {
  if (!p || T < 0 || (y_type != MOE_TYPE_BF16 && y_type != MOE_TYPE_F32)) return MOE_ERR_INVALID_ARG;
  if (T > p->T_max) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!q || !scale || !W || !W->w || !W->s || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(scale, 4) || !aligned(W->w, 256) || !aligned(W->s, 16) || !aligned(y, 16))
    return MOE_ERR_ALIGNMENT;
  if (!p->ws) return MOE_ERR_NOT_INITIALIZED;
  cudaStream_t s = S(stream);
  const int N = p->N, K = p->K, k_tiles = K / 128, m_tiles = (N + 255) / 256;
  if (linear_streams(T, k_tiles)) {
    CUtensorMap tW, tX;
    if (!make_few_maps(&tW, &tX, W->w, (uint64_t)m_tiles * k_tiles, q, T, K)) return MOE_ERR_CUDA;
    FewArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T;
    a.m_tiles = m_tiles;
    a.k_tiles = k_tiles;
    a.rows = N;
    a.sf = (const uint8_t*)W->s;
    a.xs = scale;
    a.y = y;
    a.y_f32 = y_type == MOE_TYPE_F32;
    a.part = p->at<float>(p->o_part);
    a.counters = p->at<unsigned int>(p->o_cnt);
    a.status = p->at<unsigned int>(p->o_status);
    const int grid = std::min(m_tiles * k_tiles, p->grid());
    return launch_few<FEW_LINEAR, 0>(a, tW, tX, tW, tX, grid, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  // more rows: tiles of up to 64 or 176 of them
  const LinearPick pick = pick_linear_tiles(T, m_tiles, k_tiles, p->grid());
  const int n_per = pick.n_per, n_tiles = (T + n_per - 1) / n_per;
  if ((long long)n_tiles * m_tiles * k_tiles > 0x7fffffffll || (long long)n_tiles * m_tiles > 0x7fffffffll)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  LinearArgs a;
  memset(&a, 0, sizeof(a));
  a.T = T;
  a.n_per = n_per;
  a.n_tiles = n_tiles;
  a.m_tiles = m_tiles;
  a.k_tiles = k_tiles;
  a.N = N;
  a.unit = pick.unit;
  const int units = n_tiles * m_tiles * k_tiles / a.unit;
  a.ctas = std::min(a.unit == k_tiles ? units : std::max(units / 4, 1), p->grid());
  a.per = units / a.ctas;
  a.rem = units - a.per * a.ctas;
  a.sf = (const uint8_t*)W->s;
  a.xs = scale;
  a.y = y;
  a.y_f32 = y_type == MOE_TYPE_F32;
  a.part = p->at<float>(p->o_part);
  a.status = p->at<unsigned int>(p->o_status);
  CUtensorMap tW, tX;
  if (!make_map(&tW, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, W->w, 128, (uint64_t)m_tiles * k_tiles * 256, 64, 128, 256) ||
      !make_map(&tX, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, T, K, 128, n_per))
    return MOE_ERR_CUDA;
  const cudaError_t e = n_per <= kLinearSmall ? launch_linear<kLinearSmall>(a, tW, tX, s)
                                           : launch_linear<kLinearWide>(a, tW, tX, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// ---------------------------------------------------------------- the layer for a few tokens
moe_status_t moe_forward_decode(moe_plan_t p, const void* x, const uint8_t* q, const uint8_t* scale, int T,
                                const int32_t* idx, const float* w, const moe_experts_mxfp4* ex,
                                const moe_shared_bf16* sh, void* y, void* stream) {
  if (!p || T < 0 || p->dl > 0) return MOE_ERR_INVALID_ARG;   // no latent form
  if (T > p->T_max || T > kFewRows || few_stages(FEW_GLU, T, p->k, p->d / 128) < kFewMinStages ||
      few_stages(FEW_DOWN, T, p->k, p->I / 128) < kFewMinStages ||
      (long long)p->E * (p->I / 128) * std::max(p->d / 128, (p->d + 255) / 256) * 256 > 0x7fffffffll)
    return MOE_ERR_UNSUPPORTED_SHAPE;   // (tensor-map coordinates are 32-bit)
  if (T == 0) return MOE_OK;
  if ((q != nullptr) != (scale != nullptr) || (!x && (!q || p->Is > 0))) return MOE_ERR_INVALID_ARG;
  if (!idx || !w || !ex || !y || !ex->w_gu || !ex->s_gu || !ex->w_dn || !ex->s_dn) return MOE_ERR_INVALID_ARG;
  if ((p->Is > 0) != (sh != nullptr) || (sh && (!sh->w_gu || !sh->w_dn))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4) || !aligned(y, 16) || !aligned(idx, 4) || !aligned(w, 4) ||
      !aligned(ex->w_gu, 256) || !aligned(ex->w_dn, 256) || !aligned(ex->s_gu, 16) || !aligned(ex->s_dn, 16) ||
      (sh && (!aligned(sh->w_gu, 16) || !aligned(sh->w_dn, 16))))
    return MOE_ERR_ALIGNMENT;
  if (!p->ws) return MOE_ERR_NOT_INITIALIZED;
  cudaStream_t s = S(stream);
  const int d = p->d, E = p->E, I = p->I;
  FewArgs a;
  memset(&a, 0, sizeof(a));
  a.T = T;
  a.k = p->k;
  a.E = E;
  a.idx = idx;
  a.w = w;
  a.hq = p->at<uint8_t>(p->o_fhq);
  a.hs = p->at<uint8_t>(p->o_fhs);
  a.part = p->at<float>(p->o_fpart);
  a.counters = p->at<unsigned int>(p->o_fcnt);
  a.status = p->at<unsigned int>(p->o_status);
  const int grid = std::min(p->num_sms, kFewMaxCtas);
  if (!q) {
    uint8_t* xq = p->at<uint8_t>(p->o_xq);
    uint8_t* xs = p->at<uint8_t>(p->o_xs_tok);
    p->prof.begin(MOE_STAGE_QUANT, s);
    const moe_status_t sq = moe_quant_mxfp8(x, T, d, xq, xs, stream);
    if (sq != MOE_OK) return sq;
    p->prof.end(s);
    q = xq;
    scale = xs;
  }
  CUtensorMap tW, tX, tSW, tSX;
  const int Is = p->Is;
  p->last_shared_split = p->last_shared_split_dn = 0;
  // gate/up, GLU, MXFP8 rows of the hidden values; the shared expert's hidden values
  a.m_tiles = I / 128;
  a.k_tiles = d / 128;
  a.sf = (const uint8_t*)ex->s_gu;
  a.xs = scale;
  if (!make_few_maps(&tW, &tX, ex->w_gu, (uint64_t)E * a.m_tiles * a.k_tiles, q, T, d)) return MOE_ERR_CUDA;
  tSW = tW;
  tSX = tX;
  if (sh) {
    a.sh_tiles = Is / 128;
    a.sh_steps = d / 64;
    a.hsh = p->at<__nv_bfloat16>(p->o_hsh);
    if (!make_map(&tSW, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, sh->w_gu, d, 2ull * Is, (uint64_t)d * 2, 64, 256) ||
        !make_map(&tSX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, d, T, (uint64_t)d * 2, 64, kFewRows))
      return MOE_ERR_CUDA;
  }
  p->prof.begin(MOE_STAGE_GATE_UP, s);
  if ((p->act == MOE_ACT_CLAMPED_SWIGLU ? launch_few<FEW_GLU, 1>(a, tW, tX, tSW, tSX, grid, s)
                                        : launch_few<FEW_GLU, 0>(a, tW, tX, tSW, tSX, grid, s)) != cudaSuccess)
    return MOE_ERR_CUDA;
  p->prof.end(s);
  // down products, weighted combine, the shared expert's down product
  a.m_tiles = (d + 255) / 256;
  a.k_tiles = I / 128;
  a.rows = d;
  a.sf = (const uint8_t*)ex->s_dn;
  a.y = y;
  if (!make_few_maps(&tW, &tX, ex->w_dn, (uint64_t)E * a.m_tiles * a.k_tiles, a.hq, (uint64_t)T * a.k * T, I)) return MOE_ERR_CUDA;
  if (sh) {
    a.sh_steps = Is / 64;
    if (!make_map(&tSW, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, sh->w_dn, Is, d, (uint64_t)Is * 2, 64, 256) ||
        !make_map(&tSX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.hsh, Is, T, (uint64_t)Is * 2, 64, kFewRows))
      return MOE_ERR_CUDA;
  }
  p->prof.begin(MOE_STAGE_DOWN, s);
  if (launch_few<FEW_DOWN, 0>(a, tW, tX, tSW, tSX, grid, s) != cudaSuccess) return MOE_ERR_CUDA;
  p->prof.end(s);
  p->last_T = T;
  return MOE_OK;
}

}  // extern "C"
