// Host side of the forward with an epilogue and of the grouped forward (see
// include/sbn.h): validation, the choice of kernel, the launches.

#include "sbn.h"

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "host.cuh"
#include "act_grad.cuh"
#include "bl_gemv_grp.cuh"
#include "bl_tc_grp.cuh"

namespace sbn {

sbn_status take_error_grouped(unsigned* word) { return take_error_word(g_dev_error, word); }

namespace {

// A forward over rows of one layer (offsets NULL) or of several.
struct Fwd {
  const int8_t* xq;
  const float* xs;
  const uint16_t* x;    // bf16 activations instead of xq, xs (16 rows at most)
  int8_t* xq_out;
  float* xs_out;
  GrpParams grp;
  int k, n_out, n, m;
  const uint8_t* codes;
  const uint8_t* meta;
  const float* gamma;
  EpiParams ep;
  uint16_t* y;
  int sms;
  cudaStream_t st;
  int cstride() const { return (int)sbn_codes_row_bytes(k, n, m); }
  int mstride() const { return (int)sbn_meta_row_bytes(k, n, m); }
};

template <int NT, bool XBF>
struct LaunchGemv {
  template <int MM, int CB, bool DENSE>
  static sbn_status run(const GgParams& p, int grid, cudaStream_t st) {
    static bool attr_set[kMaxDevices] = {};
    auto kern = bl_gemv_grp_kernel<MM, CB, NT, DENSE, XBF>;
    if (!set_smem_attr_once(kern, kGvSmemMax, attr_set)) return SBN_ERR_CUDA;
    return launch_ex(kern, dim3((unsigned)grid), dim3(kGvThreads), p.L.total, st, 1, p);
  }
};

// The decode kernel, where the rows fit: at most 16, their activations in the
// consumers' registers, two tiles in shared memory. false: not launched.
bool gemv_params(const Fwd& f, bool xbf, GgParams* q, int* grid) {
  const int r = f.grp.rows;
  if (r > kGgMaxRows) return false;
  const int kc = xbf ? f.k / 8 : f.k / 16;
  if ((long long)r * kc > (long long)kGvConsumers * kGvMaxChunks) return false;
  const int tpe = (f.n_out + 15) / 16;
  const long long tiles = (long long)std::min(f.grp.experts, r) * tpe;
  *grid = (int)std::min((long long)f.sms, tiles);
  const int per_cta = (int)((tiles + *grid - 1) / *grid);
  q->L = gg_layout(per_cta, r <= 8 ? 8 : 16, r, f.k, f.cstride(), f.mstride());
  if (q->L.slots == 0) return false;
  q->xq = f.xq; q->xs = f.xs; q->xbf = f.x; q->xq_out = f.xq_out; q->xs_out = f.xs_out;
  q->codes = f.codes; q->meta = f.meta; q->gamma = f.gamma; q->y = f.y; q->ep = f.ep; q->grp = f.grp;
  q->K = f.k; q->N = f.n_out; q->cstride = f.cstride(); q->mstride = f.mstride();
  q->kc = kc;
  q->kc_magic = (uint32_t)(((1ull << 32) + (unsigned long long)kc - 1) / (unsigned long long)kc);
  q->dr = kGvConsumers / kc;
  q->drem = kGvConsumers % kc;
  return true;
}

sbn_status launch_gemv_grp(const Fwd& f, bool xbf, const GgParams& q, int grid) {
  if (f.grp.rows <= 8)
    return xbf ? by_pattern<LaunchGemv<8, true>>(f.n, f.m, q, grid, f.st)
               : by_pattern<LaunchGemv<8, false>>(f.n, f.m, q, grid, f.st);
  return xbf ? by_pattern<LaunchGemv<16, true>>(f.n, f.m, q, grid, f.st)
             : by_pattern<LaunchGemv<16, false>>(f.n, f.m, q, grid, f.st);
}

struct LaunchTc {
  template <int MM, int CB, bool DENSE>
  static sbn_status run(const Fwd& f) {
    static bool attr_set[kMaxDevices] = {};
    auto kern = bl_tc_grp_kernel<MM, CB, DENSE>;
    if (!set_smem_attr_once(kern, tg_smem_bytes(kGrpMaxExperts), attr_set)) return SBN_ERR_CUDA;
    CUtensorMap x64, x16, tc, tm, ty, tz;
    if (!encode_2d(&x64, CU_TENSOR_MAP_DATA_TYPE_UINT8, f.xq, f.k, f.grp.rows, f.k, 128, 64,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&x16, CU_TENSOR_MAP_DATA_TYPE_UINT8, f.xq, f.k, f.grp.rows, f.k, 128, 16,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return SBN_ERR_CUDA;
    const uint64_t wrows = (uint64_t)f.grp.experts * (uint64_t)f.n_out;
    tm = x64;   // unused for n == m
    if (!encode_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_UINT8, f.codes, f.cstride(), wrows, f.cstride(), 16 * CB, kTgBM,
                   CU_TENSOR_MAP_SWIZZLE_NONE) ||
        (!DENSE && !encode_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, f.meta, f.mstride(), wrows, f.mstride(), 32, kTgBM,
                              CU_TENSOR_MAP_SWIZZLE_NONE)))
      return SBN_ERR_CUDA;
    TgParams p;
    p.codes = f.codes; p.meta = f.meta; p.xs = f.xs; p.gamma = f.gamma; p.y = f.y; p.ep = f.ep; p.grp = f.grp;
    p.K = f.k; p.N = f.n_out; p.cstride = f.cstride(); p.mstride = f.mstride();
    p.aligned = f.n_out % 8 == 0 && aligned16(f.y) && aligned16(f.ep.z) && aligned16(f.ep.residual);
    ty = tz = x64;   // unused unless aligned
    if (p.aligned) {
      const uint64_t pitch = 2 * (uint64_t)f.n_out;
      if (!encode_2d(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f.y, f.n_out, f.grp.rows, pitch, 32, 32,
                     CU_TENSOR_MAP_SWIZZLE_64B) ||
          (f.ep.z && !encode_2d(&tz, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f.ep.z, f.n_out, f.grp.rows, pitch, 32, 32,
                                CU_TENSOR_MAP_SWIZZLE_64B)))
        return SBN_ERR_CUDA;
    }
    // tiles: at most one more than rows / kTgBN per expert, for every block of features
    const long long row_tiles = (f.n_out + kTgBM - 1) / kTgBM;
    const long long most = (f.grp.rows / kTgBN + std::min(f.grp.experts, f.grp.rows)) * row_tiles;
    const int grid = (int)std::max(1LL, std::min(most, (long long)f.sms));
    return launch_ex(kern, dim3((unsigned)grid), dim3(kTgThreads), tg_smem_bytes(f.grp.experts), f.st, 1, x64, x16, tc,
                     tm, ty, tz, p);
  }
};

sbn_status run_grouped(const Fwd& f) {
  GgParams q;
  int grid = 0;
  if (gemv_params(f, false, &q, &grid)) return launch_gemv_grp(f, false, q, grid);
  return by_pattern<LaunchTc>(f.n, f.m, f);
}

// Checks shared by the calls (pointers of the activations apart).
sbn_status check_fwd(const Fwd& f) {
  if (!f.codes || (f.n != f.m && !f.meta) || !f.gamma || !f.y) return SBN_ERR_NULL;
  if (!pattern_ok(f.n, f.m)) return SBN_ERR_PATTERN;
  const int r = f.grp.rows, e = f.grp.experts;
  if (r < 1 || f.n_out < 1 || f.k < 128 || (f.k % 128) != 0 || e < 1 || e > kGrpMaxExperts) return SBN_ERR_SHAPE;
  if (!prod_lt_2_31(r, f.k) || !prod_lt_2_31(f.n_out, f.k) || !prod_lt_2_31(r, f.n_out) ||
      !prod_lt_2_31(e, f.n_out))
    return SBN_ERR_SHAPE;
  if (f.ep.act < 0 || f.ep.act >= kActCount) return SBN_ERR_SHAPE;
  if (!aligned16(f.codes) || !aligned16(f.meta) || !aligned16(f.y) || !aligned16(f.ep.z) || !aligned16(f.ep.residual) ||
      (reinterpret_cast<uintptr_t>(f.gamma) & 3u) || (reinterpret_cast<uintptr_t>(f.ep.bias) & 3u) ||
      (reinterpret_cast<uintptr_t>(f.grp.offsets) & 3u))
    return SBN_ERR_ALIGN;
  return SBN_OK;
}

size_t quant_bytes(int rows, int k) { return round_up16((size_t)rows * k) + round_up16((size_t)rows * 4); }

// Activation buffers of a call on bf16 activations: the given ones, or parts
// of the workspace.
void quant_buffers(int rows, int k, void* ws, int8_t** xq, float** xs) {
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  if (!*xq) *xq = reinterpret_cast<int8_t*>(w);
  if (!*xs) *xs = reinterpret_cast<float*>(w + round_up16((size_t)rows * k));
}

Fwd make_fwd(int rows, const int32_t* offsets, int experts, int k, int n_out, int n, int m, const uint8_t* codes,
             const uint8_t* meta, const float* gamma, const float* bias, int act, const void* residual, void* z,
             void* y, void* stream) {
  Fwd f = {};
  f.grp = GrpParams{offsets, experts, rows};
  f.k = k; f.n_out = n_out; f.n = n; f.m = m;
  f.codes = codes; f.meta = meta; f.gamma = gamma;
  f.ep = EpiParams{bias, reinterpret_cast<const uint16_t*>(residual), reinterpret_cast<uint16_t*>(z), act};
  f.y = reinterpret_cast<uint16_t*>(y);
  f.st = reinterpret_cast<cudaStream_t>(stream);
  return f;
}

// One layer over INT8 rows: the pair kernel where there is a workspace for
// the expanded weights, else straight from the packed ones.
sbn_status run_act(Fwd& f, void* ws) {
  if (f.grp.rows > 16 && ws) {
    const sbn_status st = run_pairs_epi(f.xq, f.xs, f.grp.rows, f.k, f.n_out, f.n, f.m, f.codes, f.meta, f.gamma, f.y,
                                        f.ep, ws, f.sms, f.st);
    if (st != SBN_ERR_DEVICE) return st;
  }
  return run_grouped(f);
}

}  // namespace
}  // namespace sbn

using namespace sbn;

extern "C" {

sbn_status sbn_bitlinear_act(const int8_t* xq, const float* x_scale, int32_t t, int32_t k, int32_t n_out, int32_t n,
                             int32_t m, const uint8_t* codes, const uint8_t* meta, const float* gamma,
                             const float* bias, int32_t act, const void* residual_bf16, void* z_bf16, void* y_bf16,
                             void* workspace, size_t ws_bytes, void* stream) {
  if (!xq || !x_scale) return SBN_ERR_NULL;
  Fwd f = make_fwd(t, nullptr, 1, k, n_out, n, m, codes, meta, gamma, bias, act, residual_bf16, z_bf16, y_bf16, stream);
  sbn_status st = check_fwd(f);
  if (st != SBN_OK) return st;
  if (!aligned16(xq) || (reinterpret_cast<uintptr_t>(x_scale) & 3u) || !aligned16(workspace)) return SBN_ERR_ALIGN;
  if (workspace && ws_bytes < sbn_bitlinear_workspace_bytes(t, k, n_out)) return SBN_ERR_WORKSPACE;
  int dev = 0;
  if ((st = check_device(&dev, &f.sms)) != SBN_OK) return st;
  f.xq = xq; f.xs = x_scale;
  return run_act(f, workspace);
}

sbn_status sbn_bitlinear_x_act(const void* x_bf16, int32_t t, int32_t k, int32_t n_out, int32_t n, int32_t m,
                               const uint8_t* codes, const uint8_t* meta, const float* gamma, const float* bias,
                               int32_t act, const void* residual_bf16, void* z_bf16, void* y_bf16, int8_t* xq,
                               float* x_scale, void* workspace, size_t ws_bytes, void* stream) {
  if (!x_bf16) return SBN_ERR_NULL;
  Fwd f = make_fwd(t, nullptr, 1, k, n_out, n, m, codes, meta, gamma, bias, act, residual_bf16, z_bf16, y_bf16, stream);
  sbn_status st = check_fwd(f);
  if (st != SBN_OK) return st;
  if (!aligned16(x_bf16) || !aligned16(xq) || (reinterpret_cast<uintptr_t>(x_scale) & 3u) || !aligned16(workspace))
    return SBN_ERR_ALIGN;
  int dev = 0;
  if ((st = check_device(&dev, &f.sms)) != SBN_OK) return st;
  f.x = reinterpret_cast<const uint16_t*>(x_bf16); f.xq_out = xq; f.xs_out = x_scale;
  GgParams q;
  int grid = 0;
  if (gemv_params(f, true, &q, &grid)) return launch_gemv_grp(f, true, q, grid);
  if (!workspace || ws_bytes < sbn_bitlinear_x_workspace_bytes(t, k, n_out)) return SBN_ERR_WORKSPACE;
  quant_buffers(t, k, workspace, &xq, &x_scale);
  if ((st = quantize_acts_rows(x_bf16, t, k, xq, x_scale, f.sms, f.st)) != SBN_OK) return st;
  f.xq = xq; f.xs = x_scale; f.x = nullptr;
  return run_act(f, reinterpret_cast<uint8_t*>(workspace) + quant_bytes(t, k));
}

sbn_status sbn_act_grad(const void* dy_bf16, const void* z_bf16, int32_t rows, const int32_t* offsets, int32_t experts,
                        int32_t n_out, int32_t act, void* dz_bf16, float* dbias, void* stream) {
  if (!dy_bf16 || !z_bf16 || !dz_bf16) return SBN_ERR_NULL;
  if (rows < 1 || n_out < 1 || experts < 1 || experts > kGrpMaxExperts || (experts > 1 && !offsets)) return SBN_ERR_SHAPE;
  if (!prod_lt_2_31(rows, n_out) || !prod_lt_2_31(experts, n_out)) return SBN_ERR_SHAPE;
  if (act < 0 || act >= kActCount) return SBN_ERR_SHAPE;
  if (!aligned16(dy_bf16) || !aligned16(z_bf16) || !aligned16(dz_bf16) || (reinterpret_cast<uintptr_t>(dbias) & 3u) ||
      (reinterpret_cast<uintptr_t>(offsets) & 3u))
    return SBN_ERR_ALIGN;
  int dev = 0, sms = 0;
  const sbn_status st = check_device(&dev, &sms);
  if (st != SBN_OK) return st;
  AgParams p;
  p.dy = reinterpret_cast<const uint16_t*>(dy_bf16); p.z = reinterpret_cast<const uint16_t*>(z_bf16);
  p.dz = reinterpret_cast<uint16_t*>(dz_bf16); p.dbias = dbias;
  p.grp = GrpParams{offsets, experts, rows}; p.N = n_out; p.act = act;
  // clusters along the rows until there are four CTAs per SM, while each has
  // a row for each of its row lanes
  const long long blocks = (long long)((n_out + kAgCols - 1) / kAgCols) * experts;
  p.cluster = 1;
  while (p.cluster < 8 && blocks * p.cluster < 4ll * sms && (long long)rows > (long long)p.cluster * kAgLanes * experts)
    p.cluster *= 2;
  const dim3 grid((unsigned)((n_out + kAgCols - 1) / kAgCols * p.cluster), (unsigned)experts);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return n_out % 8 == 0 ? launch_ex(act_grad_kernel<true>, grid, dim3(kAgThreads), 0, cs, (unsigned)p.cluster, p)
                        : launch_ex(act_grad_kernel<false>, grid, dim3(kAgThreads), 0, cs, (unsigned)p.cluster, p);
}

sbn_status sbn_bitlinear_grouped(const int8_t* xq, const float* x_scale, int32_t rows, const int32_t* offsets,
                                 int32_t experts, int32_t k, int32_t n_out, int32_t n, int32_t m,
                                 const uint8_t* codes, const uint8_t* meta, const float* gamma, const float* bias,
                                 int32_t act, const void* residual_bf16, void* z_bf16, void* y_bf16, void* stream) {
  if (!xq || !x_scale || !offsets) return SBN_ERR_NULL;
  Fwd f = make_fwd(rows, offsets, experts, k, n_out, n, m, codes, meta, gamma, bias, act, residual_bf16, z_bf16, y_bf16,
                   stream);
  sbn_status st = check_fwd(f);
  if (st != SBN_OK) return st;
  if (!aligned16(xq) || (reinterpret_cast<uintptr_t>(x_scale) & 3u)) return SBN_ERR_ALIGN;
  int dev = 0;
  if ((st = check_device(&dev, &f.sms)) != SBN_OK) return st;
  f.xq = xq; f.xs = x_scale;
  return run_grouped(f);
}

size_t sbn_bitlinear_grouped_x_workspace_bytes(int32_t rows, int32_t k) {
  return rows < 1 || k < 1 ? 0 : quant_bytes(rows, k);
}

sbn_status sbn_bitlinear_grouped_x(const void* x_bf16, int32_t rows, const int32_t* offsets, int32_t experts,
                                   int32_t k, int32_t n_out, int32_t n, int32_t m, const uint8_t* codes,
                                   const uint8_t* meta, const float* gamma, const float* bias, int32_t act,
                                   const void* residual_bf16, void* z_bf16, void* y_bf16, int8_t* xq, float* x_scale,
                                   void* workspace, size_t ws_bytes, void* stream) {
  if (!x_bf16 || !offsets) return SBN_ERR_NULL;
  Fwd f = make_fwd(rows, offsets, experts, k, n_out, n, m, codes, meta, gamma, bias, act, residual_bf16, z_bf16, y_bf16,
                   stream);
  sbn_status st = check_fwd(f);
  if (st != SBN_OK) return st;
  if (!aligned16(x_bf16) || !aligned16(xq) || (reinterpret_cast<uintptr_t>(x_scale) & 3u) || !aligned16(workspace))
    return SBN_ERR_ALIGN;
  int dev = 0;
  if ((st = check_device(&dev, &f.sms)) != SBN_OK) return st;
  f.x = reinterpret_cast<const uint16_t*>(x_bf16); f.xq_out = xq; f.xs_out = x_scale;
  GgParams q;
  int grid = 0;
  if (gemv_params(f, true, &q, &grid)) return launch_gemv_grp(f, true, q, grid);
  if ((!xq || !x_scale) && (!workspace || ws_bytes < quant_bytes(rows, k))) return SBN_ERR_WORKSPACE;
  quant_buffers(rows, k, workspace, &xq, &x_scale);
  if ((st = quantize_acts_rows(x_bf16, rows, k, xq, x_scale, f.sms, f.st)) != SBN_OK) return st;
  f.xq = xq; f.xs = x_scale; f.x = nullptr;
  return run_grouped(f);
}

}  // extern "C"
