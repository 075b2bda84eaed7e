// Host side of the grouped backward (see include/sbn.h): validation and the
// launches.

#include "sbn.h"

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "host.cuh"
#include "bwd_grp.cuh"

namespace sbn {

sbn_status take_error_grad(unsigned* word) { return take_error_word(g_dev_error, word); }

namespace {

inline int round_up8(int n) { return (n + 7) / 8 * 8; }

struct LaunchDx {
  template <int MM, int CB, bool DENSE>
  static sbn_status run(const uint16_t* dy, uint16_t* pitched, const GxParams& p, int sms, cudaStream_t st) {
    const int r = p.grp.rows, e = p.grp.experts;
    static bool attr_set[kMaxDevices] = {};
    auto kern = bwd_dx_grp_kernel<MM, CB, DENSE>;
    if (!set_smem_attr_once(kern, gx_smem_bytes(kGrpMaxExperts), attr_set)) return SBN_ERR_CUDA;
    CUtensorMap td, tc, tm;
    const uint64_t wrows = (uint64_t)e * (uint64_t)p.N;
    if (!encode_2d(&td, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pitched ? pitched : dy, round_up8(p.N), r, 2 * (uint64_t)round_up8(p.N),
                   kBxBK, kBxBM,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, p.cstride, wrows, p.cstride, 16 * CB, kBxBK,
                   CU_TENSOR_MAP_SWIZZLE_NONE))
      return SBN_ERR_CUDA;
    tm = tc;   // unused for n == m
    if (!DENSE && !encode_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.meta, p.mstride, wrows, p.mstride, 32, kBxBK,
                             CU_TENSOR_MAP_SWIZZLE_NONE))
      return SBN_ERR_CUDA;
    const long long most = (long long)(r / kBxBM + std::min(e, r)) * ((p.K + kBxBN - 1) / kBxBN);
    const int grid = (int)std::max(1LL, std::min(most, (long long)sms));
    if (pitched) {
      const long long chunks = (long long)r * (round_up8(p.N) / 8);
      const unsigned ctas = (unsigned)std::min((chunks + kGcThreads - 1) / kGcThreads, 8LL * sms);
      const sbn_status s = launch_ex(bwd_pitch_kernel, dim3(ctas), dim3(kGcThreads), 0, st, 1, dy, pitched, r, p.N);
      if (s != SBN_OK) return s;
    }
    return launch_ex(kern, dim3((unsigned)grid), dim3(kGxThreads), gx_smem_bytes(e), st, 1, td, tc, tm, p);
  }
};

// Workspace of dW: the fp16 operands over padded rows (dY s / 127 in one or two
// parts), and the scales.
struct GwLayout {
  long long rows;
  int np;
  size_t x16, scale, total;
  GwLayout(int r, int e, int k, int n, int parts) {
    rows = gw_padded_rows(r, e);
    np = round_up8(n);
    x16 = ((size_t)parts * rows * np * 2 + 127) & ~(size_t)127;
    scale = x16 + (((size_t)rows * k * 2 + 127) & ~(size_t)127);
    total = scale + round_up16((size_t)e * n * 4);
  }
};

template <int PARTS>
sbn_status launch_dw(const GwParams& p, const GwLayout& l, int grid, cudaStream_t st) {
  const int e = p.grp.experts;
  CUtensorMap ta, tx, tdw;
  if (!encode_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.a16, l.np, (uint64_t)PARTS * l.rows, 2 * (uint64_t)l.np, 64,
                 kGwBK, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.x16, p.K, l.rows, 2 * (uint64_t)p.K, 64, kGwBK,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tdw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.dw, p.K, (uint64_t)e * (uint64_t)p.N, 2 * (uint64_t)p.K, 32, 32,
                 CU_TENSOR_MAP_SWIZZLE_64B))
    return SBN_ERR_CUDA;
  static bool attr_set[kMaxDevices] = {};
  if (!set_smem_attr_once(bwd_dw_grp_kernel<PARTS>, gw_smem_bytes(kGrpMaxExperts), attr_set)) return SBN_ERR_CUDA;
  return launch_ex(bwd_dw_grp_kernel<PARTS>, dim3((unsigned)grid), dim3(kGwThreads), gw_smem_bytes(e), st, 1, ta, tx, tdw,
                   p);
}

sbn_status check_grad(int rows, const int32_t* offsets, int experts, int k, int n_out) {
  if (rows < 1 || n_out < 1 || k < 128 || (k % 128) != 0 || experts < 1 || experts > kGrpMaxExperts) return SBN_ERR_SHAPE;
  if (!prod_lt_2_31(rows, k) || !prod_lt_2_31(n_out, k) || !prod_lt_2_31(rows, n_out) ||
      !prod_lt_2_31(experts, n_out))
    return SBN_ERR_SHAPE;
  return (reinterpret_cast<uintptr_t>(offsets) & 3u) ? SBN_ERR_ALIGN : SBN_OK;
}

}  // namespace
}  // namespace sbn

using namespace sbn;

extern "C" {

size_t sbn_bitlinear_grouped_grad_x_workspace_bytes(int32_t rows, int32_t n_out) {
  if (rows < 1 || n_out < 1 || !prod_lt_2_31(rows, n_out) || n_out % 8 == 0) return 0;
  return (size_t)rows * round_up8(n_out) * 2;
}

sbn_status sbn_bitlinear_grouped_grad_x(const void* dy_bf16, int32_t rows, const int32_t* offsets, int32_t experts,
                                        int32_t k, int32_t n_out, int32_t n, int32_t m, const uint8_t* codes,
                                        const uint8_t* meta, const float* gamma, void* dx_bf16, void* workspace,
                                        size_t ws_bytes, void* stream) {
  if (!dy_bf16 || !offsets || !codes || !gamma || !dx_bf16 || (n != m && !meta)) return SBN_ERR_NULL;
  if (!pattern_ok(n, m)) return SBN_ERR_PATTERN;
  sbn_status st = check_grad(rows, offsets, experts, k, n_out);
  if (st != SBN_OK) return st;
  if (!aligned16(dy_bf16) || !aligned16(codes) || !aligned16(meta) || !aligned16(dx_bf16) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(gamma) & 3u))
    return SBN_ERR_ALIGN;
  const size_t need = sbn_bitlinear_grouped_grad_x_workspace_bytes(rows, n_out);
  if (need && (!workspace || ws_bytes < need)) return SBN_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != SBN_OK) return st;
  GxParams p;
  p.codes = codes; p.meta = meta; p.gamma = gamma; p.dx = reinterpret_cast<uint16_t*>(dx_bf16);
  p.grp = GrpParams{offsets, experts, rows}; p.K = k; p.N = n_out;
  p.cstride = (int)sbn_codes_row_bytes(k, n, m); p.mstride = (int)sbn_meta_row_bytes(k, n, m);
  return by_pattern<LaunchDx>(n, m, reinterpret_cast<const uint16_t*>(dy_bf16),
                              need ? reinterpret_cast<uint16_t*>(workspace) : nullptr, p, sms,
                              reinterpret_cast<cudaStream_t>(stream));
}

size_t sbn_bitlinear_grouped_grad_w_workspace_bytes(int32_t rows, int32_t experts, int32_t k, int32_t n_out) {
  if (check_grad(rows, nullptr, experts, k, n_out) != SBN_OK) return 0;
  return GwLayout(rows, experts, k, n_out, 1).total;
}

size_t sbn_bitlinear_grouped_grad_w2_workspace_bytes(int32_t rows, int32_t experts, int32_t k, int32_t n_out) {
  if (check_grad(rows, nullptr, experts, k, n_out) != SBN_OK) return 0;
  return GwLayout(rows, experts, k, n_out, 2).total;
}

sbn_status sbn_bitlinear_grouped_grad_w(const void* dy_bf16, const int8_t* xq, const float* x_scale, int32_t rows,
                                        const int32_t* offsets, int32_t experts, int32_t k, int32_t n_out,
                                        void* dw_bf16, void* workspace, size_t ws_bytes, void* stream) {
  if (!dy_bf16 || !xq || !x_scale || !offsets || !dw_bf16) return SBN_ERR_NULL;
  sbn_status st = check_grad(rows, offsets, experts, k, n_out);
  if (st != SBN_OK) return st;
  if (!aligned16(dy_bf16) || !aligned16(xq) || !aligned16(dw_bf16) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(x_scale) & 3u))
    return SBN_ERR_ALIGN;
  const size_t need = sbn_bitlinear_grouped_grad_w_workspace_bytes(rows, experts, k, n_out);
  if (!workspace || ws_bytes < need) return SBN_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != SBN_OK) return st;
  GwParams p = {};
  p.dy = reinterpret_cast<const uint16_t*>(dy_bf16); p.xq = xq; p.xs = x_scale;
  p.dw = reinterpret_cast<uint16_t*>(dw_bf16); p.grp = GrpParams{offsets, experts, rows}; p.K = k; p.N = n_out;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const size_t list = 8 * (size_t)(experts + 1);
  const int parts = ws_bytes >= sbn_bitlinear_grouped_grad_w2_workspace_bytes(rows, experts, k, n_out) ? 2 : 1;
  const GwLayout l(rows, experts, k, n_out, parts);
  uint8_t* w8 = reinterpret_cast<uint8_t*>(workspace);
  p.Np = l.np;
  p.a_rows = parts == 2 ? l.rows : 0;
  p.a16 = reinterpret_cast<uint16_t*>(w8);
  p.x16 = reinterpret_cast<uint16_t*>(w8 + l.x16);
  p.scale = reinterpret_cast<float*>(w8 + l.scale);
  // the preparation: clusters along an expert's rows until four CTAs per SM
  // scale dY, and as many CTAs again for Xq
  const long long blocks = (long long)((n_out + kGpCols - 1) / kGpCols) * experts;
  p.cluster = 1;
  while (p.cluster < 8 && blocks * p.cluster < 4ll * sms && (long long)rows > 2ll * p.cluster * kGpLanes * experts)
    p.cluster *= 2;
  if (blocks * p.cluster > (1ll << 30)) return SBN_ERR_SHAPE;
  p.a_ctas = (int)(blocks * p.cluster);
  const int x_ctas = std::min(4 * sms, (int)((l.rows + 7) / 8));
  const unsigned grid = (unsigned)((p.a_ctas + x_ctas + p.cluster - 1) / p.cluster * p.cluster);
  const auto prep = n_out % 8 == 0 ? bwd_dw_prep_kernel<true> : bwd_dw_prep_kernel<false>;
  if ((st = launch_ex(prep, dim3(grid), dim3(kGpThreads), list, cs, (unsigned)p.cluster, p)) != SBN_OK)
    return st;
  const long long tiles = (long long)experts * ((n_out + kGwBM - 1) / kGwBM) * ((k + kGwBN - 1) / kGwBN);
  const int main_grid = (int)std::min(tiles, (long long)sms);
  return parts == 2 ? launch_dw<2>(p, l, main_grid, cs) : launch_dw<1>(p, l, main_grid, cs);
}

}  // extern "C"
