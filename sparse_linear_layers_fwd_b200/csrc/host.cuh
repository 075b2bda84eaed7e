// Host helpers shared by the library's translation units: argument and
// device checks, launches with the programmatic attribute, the tensor-map
// encoder. One copy of each piece of state serves every unit.
#pragma once

#include "sbn.h"

#include <atomic>
#include <cstdint>
#include <utility>

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace sbn {

constexpr int kMaxDevices = 64;
inline int g_dev_checked[kMaxDevices];  // 0 unknown, 1 ok, -1 unsupported
inline int g_dev_sms[kMaxDevices];

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0u; }

inline bool pattern_ok(int n, int m) {
  return (m == 4 || m == 8 || m == 16) && n >= 1 && n <= m && (4 * n) % m == 0;
}

inline bool prod_lt_2_31(long long a, long long b) { return a >= 0 && b >= 0 && a * b < (1ll << 31); }

inline size_t round_up16(size_t x) { return (x + 15u) & ~size_t(15); }

// Current device must be an sm_100 part (the library carries sm_100a code only).
inline sbn_status check_device(int* dev_out, int* sms_out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return SBN_ERR_CUDA; }
  if (dev < 0 || dev >= kMaxDevices) return SBN_ERR_DEVICE;
  if (g_dev_checked[dev] == 0) {
    int major = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return SBN_ERR_CUDA;
    }
    g_dev_sms[dev] = sms;
    g_dev_checked[dev] = (major == 10) ? 1 : -1;
  }
  if (g_dev_checked[dev] < 0) return SBN_ERR_DEVICE;
  *dev_out = dev;
  *sms_out = g_dev_sms[dev];
  return SBN_OK;
}

inline sbn_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? SBN_OK : SBN_ERR_CUDA;
}

// Programmatic dependent launch of the kernels that call griddep_wait()
// before touching global memory: each may be scheduled while the previous
// grid on the stream is finishing, so its launch and set-up (barriers,
// TMEM, selector tables) overlap that grid's tail. Switched by
// sbn_set_programmatic_launch; on by default.
inline std::atomic<int> g_pdl{1};

// The dynamic shared-memory limit of a kernel, raised once per device (flags:
// one per device, owned by the caller's instantiation).
template <typename K>
bool set_smem_attr_once(K kern, size_t bytes, bool* flags) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return false;
  }
  if (!flags[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    flags[dev] = true;
  }
  return true;
}

// cudaLaunchKernelEx with the programmatic attribute (when switched on) and,
// for cluster > 1, clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
sbn_status launch_ex(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                     unsigned cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (g_pdl.load(std::memory_order_relaxed)) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  if (cluster > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = cluster;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  if (cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return SBN_ERR_CUDA;
  }
  return SBN_OK;
}

// cuTensorMapEncodeTiled from the driver, looked up once (no libcuda link).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// Calls F::run<m, code bytes per 16 positions, n == m> for the pattern.
template <typename F, typename... Args>
sbn_status by_pattern(int n, int m, Args&&... args) {
  if (n == m) return F::template run<8, 4, true>(std::forward<Args>(args)...);
  switch (m * 8 + 4 * n / m) {
    case 4 * 8 + 1: return F::template run<4, 1, false>(std::forward<Args>(args)...);
    case 4 * 8 + 2: return F::template run<4, 2, false>(std::forward<Args>(args)...);
    case 4 * 8 + 3: return F::template run<4, 3, false>(std::forward<Args>(args)...);
    case 8 * 8 + 1: return F::template run<8, 1, false>(std::forward<Args>(args)...);
    case 8 * 8 + 2: return F::template run<8, 2, false>(std::forward<Args>(args)...);
    case 8 * 8 + 3: return F::template run<8, 3, false>(std::forward<Args>(args)...);
    case 16 * 8 + 1: return F::template run<16, 1, false>(std::forward<Args>(args)...);
    case 16 * 8 + 2: return F::template run<16, 2, false>(std::forward<Args>(args)...);
    case 16 * 8 + 3: return F::template run<16, 3, false>(std::forward<Args>(args)...);
  }
  return SBN_ERR_PATTERN;
}

// Tensor map of a row-major matrix (rows of row_bytes bytes).
inline bool encode_2d(CUtensorMap* tm, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows,
               uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t gdim[2] = {inner, rows};
  cuuint64_t gstride[1] = {row_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estride[2] = {1, 1};
  return enc(tm, type, 2, const_cast<void*>(base), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct EpiParams;   // epi.cuh

// Calls across the units. quantize_acts_rows: sbn_quantize_acts after its
// checks. run_pairs_epi: t > 16 rows through the CTA-pair kernel with the
// epilogue, ws as for sbn_bitlinear; SBN_ERR_DEVICE before any launch where no
// pair can be resident.
sbn_status quantize_acts_rows(const void* x_bf16, int t, int k, int8_t* xq, float* x_scale, int sms, cudaStream_t s);
sbn_status run_pairs_epi(const int8_t* xq, const float* xs, int t, int k, int n_out, int n, int m, const uint8_t* codes,
                         const uint8_t* meta, const float* gamma, uint16_t* y, const EpiParams& ep, void* ws, int sms,
                         cudaStream_t st);

// Device error words of the translation units (common.cuh): each unit reads
// its own and clears it. 0: none; a CUDA failure is reported as such.
sbn_status take_error_grouped(unsigned* word);
sbn_status take_error_grad(unsigned* word);

template <typename Sym>
sbn_status take_error_word(const Sym& sym, unsigned* word) {
  const unsigned zero = 0u;
  if (cudaMemcpyFromSymbol(word, sym, sizeof(unsigned)) != cudaSuccess ||
      cudaMemcpyToSymbol(sym, &zero, sizeof(zero)) != cudaSuccess) {
    cudaGetLastError();
    return SBN_ERR_CUDA;
  }
  return SBN_OK;
}

}  // namespace sbn
