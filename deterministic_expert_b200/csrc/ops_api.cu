// C entry points of the handle-free expert-layer operators (include/moe.h).
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "moe_internal.h"
#include "ops_internal.h"

using namespace moe;

namespace {

// Rows (and columns) that the kernels' 32-bit indexes can round up to whole tiles.
constexpr int kMost = INT_MAX - 256;

bool al(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
size_t dtype_size(int d) { return d == MOE_DTYPE_BF16 ? 2 : 4; }
int status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();   // the failure is reported here, not by the next call
  return MOE_ECUDA;
}

PFN_cuTensorMapEncodeTiled_v12000 encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// E4M3 bytes [outer, rows, inner] (outer = 0: [rows, inner]), boxes of 128 codes x
// box_rows rows with 128-byte swizzling; what lies outside reads as zeros.
bool code_map(CUtensorMap* m, const void* p, uint64_t inner, uint64_t rows, uint64_t outer, uint32_t box_rows) {
  auto fn = encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {inner, rows, outer};
  const cuuint64_t strides[2] = {inner, inner * rows};
  const cuuint32_t box[3] = {128, box_rows, 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, outer ? 3 : 2, const_cast<void*>(p), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_route(const moe_route_config* c, int T) {
  if (!c || T < 0 || c->E <= 0 || c->k <= 0 || c->n_groups <= 0 || c->topk_groups <= 0 ||
      c->topk_groups > c->n_groups || (c->group_top != 1 && c->group_top != 2) || !dtype_ok(c->logits_dtype) ||
      (c->scores != MOE_ROUTER_SOFTMAX && c->scores != MOE_ROUTER_SIGMOID_BIAS) || std::isnan(c->routed_scale))
    return MOE_EINVAL;
  if (c->E > kRouteMaxE || c->k > kRouteMaxK || c->k > c->E || c->n_groups > 32 || c->E % c->n_groups)
    return MOE_EUNSUPPORTED;
  if (static_cast<long long>(T) * c->k > kMost) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_glu(const moe_glu_config* c) {
  if (!c) return MOE_EINVAL;
  if (c->activation == MOE_ACT_SWIGLU)
    return c->gate_clamp_max > -INFINITY && c->up_clamp >= 0.f ? MOE_OK : MOE_EINVAL;
  if (c->activation == MOE_ACT_SITU_GLU)
    return c->situ_beta_gate > 0.f && std::isfinite(c->situ_beta_gate) && c->situ_beta_up > 0.f &&
                   std::isfinite(c->situ_beta_up)
               ? MOE_OK
               : MOE_EINVAL;
  return MOE_EINVAL;
}

// A row pitch in elements whose rows all start on 16 bytes.
bool pitch16(long long ld, size_t size) { return (static_cast<unsigned long long>(ld) * size) % 16 == 0; }

}  // namespace

extern "C" {

int moe_route(const moe_route_config* cfg, int T, const void* logits, long long ld, const float* bias,
              int32_t* out_idx, float* out_w, void* stream) {
  const int v = check_route(cfg, T);
  if (v != MOE_OK) return v;
  RouteOpArgs a = {};
  a.gs = cfg->E / cfg->n_groups;
  a.lpg = 1;
  while (a.lpg * 2 * cfg->n_groups <= 32) a.lpg *= 2;
  a.cpl = (a.gs + a.lpg - 1) / a.lpg;
  if (a.cpl > kRouteMaxPerLane) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  const size_t size = dtype_size(cfg->logits_dtype);
  if (!logits || !out_idx || !out_w || ld < cfg->E || !al(logits, size) || !al(bias, 4) || !al(out_idx, 4) ||
      !al(out_w, 4))
    return MOE_EINVAL;
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.T = T;
  a.E = cfg->E;
  a.k = cfg->k;
  a.softmax = cfg->scores == MOE_ROUTER_SOFTMAX;
  a.n_groups = cfg->n_groups;
  a.topk_groups = cfg->topk_groups;
  a.group_top = cfg->group_top;
  a.renorm = cfg->renormalize != 0;
  a.scale = cfg->routed_scale;
  a.idx = out_idx;
  a.w = out_w;
  a.vec = a.cpl * a.lpg == a.gs && (a.cpl * size) % 16 == 0 && al(logits, 16) && pitch16(ld, size);
  a.vec_bias = a.cpl * a.lpg == a.gs && a.cpl % 4 == 0 && al(bias, 16);
  return status(launch_route(a, cfg->logits_dtype == MOE_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

int moe_route_backward(const moe_route_config* cfg, int T, const void* logits, long long ld, const int32_t* idx,
                       const float* dw, void* dlogits, long long ld_out, void* stream) {
  const int v = check_route(cfg, T);
  if (v != MOE_OK) return v;
  if (T == 0) return MOE_OK;
  const size_t size = dtype_size(cfg->logits_dtype);
  if (!logits || !idx || !dw || !dlogits || ld < cfg->E || ld_out < cfg->E || !al(logits, size) ||
      !al(dlogits, size) || !al(idx, 4) || !al(dw, 4))
    return MOE_EINVAL;
  RouteBackArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.idx = idx;
  a.dw = dw;
  a.dlogits = dlogits;
  a.ld_out = ld_out;
  a.T = T;
  a.E = cfg->E;
  a.k = cfg->k;
  a.softmax = cfg->scores == MOE_ROUTER_SOFTMAX;
  a.renorm = cfg->renormalize != 0;
  a.scale = cfg->routed_scale;
  a.vec = cfg->E % 4 == 0 && ld % 4 == 0 && ld_out % 4 == 0 && al(logits, 4 * size) && al(dlogits, 4 * size);
  return status(launch_route_backward(a, cfg->logits_dtype == MOE_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

int moe_group_rows(int T, int k, int E, const int32_t* idx, int32_t* offsets, int32_t* token_of_row,
                   int32_t* row_of_slot, void* stream) {
  if (T < 0 || k <= 0 || E <= 0 || !offsets || !al(offsets, 4)) return MOE_EINVAL;
  if (E > kRouteMaxE || static_cast<long long>(T) * k > kMost) return MOE_EUNSUPPORTED;
  if (T > 0 && (!idx || !token_of_row || !row_of_slot || !al(idx, 4) || !al(token_of_row, 4) || !al(row_of_slot, 4)))
    return MOE_EINVAL;
  // T = 0 still writes the offsets (all 0).
  return status(launch_group_rows(idx, T, k, E, offsets, token_of_row, row_of_slot, static_cast<cudaStream_t>(stream)));
}

int moe_quantize_rows_fp8(int rows, int K, const void* x, int dtype, long long ld, int src_rows,
                          const int32_t* token_of_row, const int32_t* n_rows, uint8_t* codes, float* scales,
                          long long ld_s, void* stream) {
  if (rows < 0 || K <= 0 || !dtype_ok(dtype) || src_rows < 0) return MOE_EINVAL;
  if (K % 16 || K > (1 << 20) || rows > kMost) return MOE_EUNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || ld < K || ld_s < rows || !al(x, 16) || !pitch16(ld, dtype_size(dtype)) ||
      !al(codes, 16) || !al(scales, 4) || !al(token_of_row, 4) || !al(n_rows, 4))
    return MOE_EINVAL;
  QuantArgs a = {};
  a.x = x;
  a.ld = ld;
  a.token_of_row = token_of_row;
  a.src_rows = src_rows;
  a.n_rows = n_rows;
  a.R = rows;
  a.K = K;
  a.codes = codes;
  a.scales = scales;
  a.ld_s = ld_s;
  return status(launch_quant_blocks(a, dtype == MOE_DTYPE_BF16 ? kQuantBf16 : kQuantF32,
                                    static_cast<cudaStream_t>(stream)));
}

int moe_quantize_weights_fp8(int G, int N, int K, const moe_bf16* w, uint8_t* codes, float* scales, void* stream) {
  if (G < 0 || N <= 0 || K <= 0) return MOE_EINVAL;
  if (K % 16 || K > kMost || G > 65535 || (N + 127ll) / 128 > 65535) return MOE_EUNSUPPORTED;
  if (G == 0) return MOE_OK;
  if (!w || !codes || !scales || !al(w, 16) || !al(codes, 16) || !al(scales, 4)) return MOE_EINVAL;
  return status(launch_quant_weights_block(w, codes, scales, G, N, K, static_cast<cudaStream_t>(stream)));
}

static int glu_args(const moe_glu_config* cfg, int rows, int I, const moe_bf16* gu, long long ld,
                    const int32_t* n_rows, uint8_t* codes, float* scales, long long ld_s, QuantArgs* a) {
  const int v = check_glu(cfg);
  if (v != MOE_OK) return v;
  if (rows < 0 || I <= 0) return MOE_EINVAL;
  if (I % 16 || I > (1 << 19) || rows > kMost) return MOE_EUNSUPPORTED;
  if (rows > 0 && (!gu || !codes || !scales || ld < 2ll * I || ld_s < rows || !al(gu, 16) || !pitch16(ld, 2) ||
                   !al(codes, 16) || !al(scales, 4) || !al(n_rows, 4)))
    return MOE_EINVAL;
  *a = {};
  a->x = gu;
  a->ld = ld;
  a->n_rows = n_rows;
  a->R = rows;
  a->K = I;
  a->codes = codes;
  a->scales = scales;
  a->ld_s = ld_s;
  a->act = cfg->activation;
  a->clamped = std::isfinite(cfg->gate_clamp_max) || std::isfinite(cfg->up_clamp);
  a->gate_clamp = cfg->gate_clamp_max;
  a->up_clamp = cfg->up_clamp;
  a->beta_g = cfg->situ_beta_gate;
  a->beta_u = cfg->situ_beta_up;
  return MOE_OK;
}

int moe_glu_quantize_fp8(const moe_glu_config* cfg, int rows, int I, const moe_bf16* gu, long long ld,
                         const int32_t* n_rows, uint8_t* codes, float* scales, long long ld_s, void* stream) {
  QuantArgs a;
  const int v = glu_args(cfg, rows, I, gu, ld, n_rows, codes, scales, ld_s, &a);
  if (v != MOE_OK || rows == 0) return v;
  return status(launch_quant_blocks(a, kQuantGlu, static_cast<cudaStream_t>(stream)));
}

int moe_glu_backward_quantize_fp8(const moe_glu_config* cfg, int rows, int I, const moe_bf16* gu, long long ld,
                                  const moe_bf16* dh, long long ld_dh, const int32_t* n_rows, uint8_t* codes,
                                  float* scales, long long ld_s, void* stream) {
  QuantArgs a;
  const int v = glu_args(cfg, rows, I, gu, ld, n_rows, codes, scales, ld_s, &a);
  if (v != MOE_OK) return v;
  if (I % 128) return MOE_EUNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!dh || ld_dh < I || !al(dh, 16) || !pitch16(ld_dh, 2)) return MOE_EINVAL;
  a.dh = dh;
  a.ld_dh = ld_dh;
  return status(launch_quant_blocks(a, kQuantGluBackward, static_cast<cudaStream_t>(stream)));
}

// Tries of a bounded wait, of up to about a microsecond each.
constexpr int kTries = 4 << 20;

// load_blocks: blocks of the contraction that are loaded, below all of them only in
// the waits' self-test.
static int matmul(int transposed, int G, const int32_t* offsets, int M, int N, int K, const uint8_t* a,
                  const float* a_scale, long long ld_as, const uint8_t* w, const float* w_scale, void* out,
                  int out_dtype, long long ldo, int load_blocks, int tries, void* stream) {
  if (G <= 0 || M < 0 || N <= 0 || K <= 0 || !dtype_ok(out_dtype) || (transposed != 0 && transposed != 1) ||
      (G > 1 && M > 0 && !offsets))
    return MOE_EINVAL;
  if (K % 16 || (transposed && N % 16) || G > kMatmulMaxGroups || M > kMost || N > kMost || K > kMost)
    return MOE_EUNSUPPORTED;
  if (M == 0) return MOE_OK;
  const int con = transposed ? N : K, width = transposed ? K : N;
  const size_t osize = dtype_size(out_dtype);
  const long long ntn = (width + 255) / 256;
  // Rows per tile.  256 rows run as full tiles; where groups are small (at most a
  // quarter of that on average, so that few have a second tile) or, below, the tiles
  // too few for the device's CTA pairs, less.  No choice changes a result's bits.
  const long long avg = (static_cast<long long>(M) + G - 1) / G;
  const long long rows_most = std::min<long long>(M, 4 * avg);
  int tr = 256;
  while (tr > 32 && tr / 2 >= rows_most) tr /= 2;
  // Tiles are counted in 32 bits on the device, whatever the offsets hold there.
  if (static_cast<double>(ntn) * ((M + tr - 1ll) / tr) * G > 0x7fff0000) return MOE_EUNSUPPORTED;
  if (!a || !a_scale || !w || !w_scale || !out || ld_as < M || ldo < width || !al(a, 16) || !al(w, 16) ||
      !al(a_scale, 4) || !al(w_scale, 4) || !al(out, osize) || !al(offsets, 4))
    return MOE_EINVAL;
  const int pairs = block_gemm_pairs();
  if (pairs <= 0) return status(cudaErrorInvalidConfiguration);

  BlockGemmArgs g = {};
  auto tiles = [&](int rows) { return ntn * std::max<long long>((M + rows - 1) / rows, std::min(G, M)); };
  while (tr > 32 && tiles(tr) < pairs) tr /= 2;
  // At most 32 rows, and too few tiles for the SMs: clusters of 2 or 4 CTAs share a
  // tile's contraction (tiles of 128 columns).  Each CTA in the walk costs about
  // 1.5 us, so 4 only for 32 blocks or more; 8 lost everywhere, as few clusters of 8
  // fit the device at once.  The block sums of a CTA's run have to fit 512 TMEM
  // columns.  Measured, us (pair tiles; 2; 4): M = 8, N = 4096, K = 7168: 20; 15.2;
  // 13.3.  M = 32: 21.5; not; 17.5.  M = 16, N = 7168, K = 2048: 9.5; 7.9; 16.1.
  const int thin_rows = M <= 16 ? 16 : 32;
  const long long thin_tiles = (width + 127ll) / 128 * std::min(G, M);   // one a group with rows
  const long long nkb = (con + 127ll) / 128;
  int split = 0;
  if (M <= 32 && nkb >= 8 && thin_tiles <= pairs) {
    const bool four = thin_tiles * 4 <= 128;
    split = four && (nkb >= 32 || (nkb + 1) / 2 * thin_rows > 512) ? 4 : 2;
    if ((nkb + split - 1) / split * thin_rows > 512) split = 0;
  }
  if (split) tr = thin_rows;
  const int per_cta = split ? tr : (tr == 256 ? 128 : tr / 2);
  int boxes = 1;
  while ((16 << (boxes - 1)) < per_cta) ++boxes;
  for (int b = 0; b < boxes; ++b)
    if (!code_map(&g.mapA[b], a, con, M, 0, 16u << b)) return status(cudaErrorInvalidValue);
  if (!code_map(&g.mapW, w, K, N, G, 128)) return status(cudaErrorInvalidValue);
  g.offsets = offsets;
  g.G = G;
  g.M = M;
  g.con = con;
  g.width = width;
  g.transposed = transposed;
  g.tile_rows = tr;
  g.split = split;
  g.a_slot = (16 << (boxes - 1)) * 128;
  g.a_scale = a_scale;
  g.ld_as = ld_as;
  g.w_scale = w_scale;
  const long long nb = (N + 127) / 128, kb = (K + 127) / 128;
  g.ws_g = nb * kb;
  g.ws_o = transposed ? 1 : kb;
  g.ws_c = transposed ? kb : 1;
  g.out = out;
  g.ldo = ldo;
  g.out_f32 = out_dtype == MOE_DTYPE_F32;
  g.out_vec = al(out, 16) && pitch16(ldo, osize);
  g.load_blocks = static_cast<int>(std::min<long long>(nkb, load_blocks));
  g.tries = tries;
  const long long max_tiles = split ? thin_tiles : std::min<long long>(ntn * ((M + tr - 1) / tr + G), pairs);
  return status(launch_block_gemm(g, static_cast<int>(max_tiles),
                                  static_cast<cudaStream_t>(stream)));
}

int moe_matmul_fp8(int transposed, int G, const int32_t* offsets, int M, int N, int K, const uint8_t* a,
                   const float* a_scale, long long ld_as, const uint8_t* w, const float* w_scale, void* out,
                   int out_dtype, long long ldo, void* stream) {
  return matmul(transposed, G, offsets, M, N, K, a, a_scale, ld_as, w, w_scale, out, out_dtype, ldo, INT_MAX, kTries,
                stream);
}

int moe_selftest_matmul_timeout(int M, int N, int K, int load_blocks, void* stream) {
  if (M < 1 || M > 8192 || N < 1 || N > 8192 || K < 1 || K > 8192 || load_blocks < 0) return MOE_EINVAL;
  if (K % 16) return MOE_EUNSUPPORTED;
  // Rows, weights, their scales, the product: all zeros.
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t kb = (K + 127) / 128, nb = (N + 127) / 128;
  const size_t sizes[5] = {up(size_t(M) * K), up(size_t(N) * K), up(kb * M * 4), up(nb * kb * 4), up(size_t(M) * N * 4)};
  size_t at[6] = {};
  for (int i = 0; i < 5; ++i) at[i + 1] = at[i] + sizes[i];
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* p = nullptr;
  if (cudaMalloc(&p, at[5]) != cudaSuccess) return status(cudaErrorMemoryAllocation);
  int res = status(cudaMemsetAsync(p, 0, at[5], s));
  if (res == MOE_OK)
    res = matmul(0, 1, nullptr, M, N, K, p, reinterpret_cast<float*>(p + at[2]), M, p + at[1],
                 reinterpret_cast<float*>(p + at[3]), p + at[4], MOE_DTYPE_F32, N, load_blocks, 1 << 14, s);
  if (res == MOE_OK) res = moe_get_operator_error(s);   // synchronises
  cudaStreamSynchronize(s);
  cudaFree(p);
  return res;
}

int moe_combine_rows(int T, int k, int D, int rows, const void* y, int y_dtype, long long ld_y,
                     const int32_t* row_of_slot, const float* w, const moe_bf16* addend, void* out, int out_dtype,
                     void* stream) {
  if (T < 0 || k <= 0 || D <= 0 || rows < 0 || !dtype_ok(y_dtype) || !dtype_ok(out_dtype)) return MOE_EINVAL;
  if (D % 8 || k > kRouteMaxK || D > (1 << 20) || T > kMost || rows > kMost) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!row_of_slot || !out || (rows > 0 && !y) || ld_y < D || !al(y, 16) || !pitch16(ld_y, dtype_size(y_dtype)) ||
      !al(row_of_slot, 4) || !al(w, 4) || !al(addend, 16) || !al(out, 16))
    return MOE_EINVAL;
  CombineArgs a = {};
  a.y = y;
  a.ld_y = ld_y;
  a.rows = rows;
  a.row_of_slot = row_of_slot;
  a.w = w;
  a.addend = addend;
  a.T = T;
  a.k = k;
  a.D = D;
  a.out = out;
  return status(launch_combine_rows(a, y_dtype == MOE_DTYPE_F32, out_dtype == MOE_DTYPE_F32,
                                    static_cast<cudaStream_t>(stream)));
}

int moe_combine_rows_backward(int T, int k, int D, int rows, const moe_bf16* dout, const void* y, int y_dtype,
                              long long ld_y, const int32_t* row_of_slot, const float* w, void* dy, float* dw,
                              void* stream) {
  if (T < 0 || k <= 0 || D <= 0 || rows < 0 || !dtype_ok(y_dtype)) return MOE_EINVAL;
  if (D % 8 || k > kRouteMaxK || D > (1 << 20) || T > kMost || rows > kMost) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dout || !row_of_slot || (rows > 0 && (!dy || (dw && !y))) || ld_y < D || !al(dout, 16) || !al(y, 16) ||
      !pitch16(ld_y, dtype_size(y_dtype)) || !al(row_of_slot, 4) || !al(w, 4) || !al(dy, 16) || !al(dw, 4))
    return MOE_EINVAL;
  CombineArgs a = {};
  a.y = y;
  a.ld_y = ld_y;
  a.rows = rows;
  a.row_of_slot = row_of_slot;
  a.w = w;
  a.T = T;
  a.k = k;
  a.D = D;
  a.dout = dout;
  a.dy = dy;
  a.dw = dw;
  return status(launch_combine_rows_backward(a, y_dtype == MOE_DTYPE_F32, static_cast<cudaStream_t>(stream)));
}

int moe_get_operator_error(void* stream) {
  int v = 0;
  if (read_operator_error(&v, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ECUDA;
  }
  return v == 0 ? MOE_OK : (v == 1 ? MOE_ETIMEOUT : (v == 3 ? MOE_EINDEX : MOE_ECUDA));
}

}  // extern "C"
