// Host side of sbn_adamw (see include/sbn.h): validation, the tensor table,
// the launches.

#include "sbn.h"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "host.cuh"
#include "adamw.cuh"

namespace sbn {
namespace {

constexpr int kAwSmall = 24, kAwLarge = 440;   // table sizes (kernel parameters end at 32764 bytes)
static_assert(sizeof(AwTable<kAwLarge>) + sizeof(AwHyper) < 32000, "kernel parameters");

template <typename P, typename G, int BITS, int N>
sbn_status launch_adamw(const sbn_adamw_tensor* t, int count, uint32_t id0, bool last, const AwHyper& hp, int sms,
                        cudaStream_t st) {
  static int cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return SBN_ERR_CUDA;
  }
  auto kern = adamw_kernel<P, G, BITS, N>;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kAwThreads, 0) != cudaSuccess || n < 1) n = 1;
    cudaGetLastError();
    cache[dev] = n;
  }
  AwTable<N> tab;
  uint32_t at = 0;
  const uintptr_t s_mask = BITS == 32 ? 31u : 7u;
  for (int i = 0; i < count; ++i) {
    AwEntry& e = tab.e[i];
    e.p = t[i].p; e.g = t[i].g; e.m = t[i].m; e.v = t[i].v;
    e.ms = t[i].m_scale; e.vs = t[i].v_scale; e.copy = reinterpret_cast<uint16_t*>(t[i].copy_bf16);
    e.numel = (uint32_t)t[i].numel;
    const uintptr_t bad = (reinterpret_cast<uintptr_t>(e.p) & (8 * sizeof(P) - 1)) |
                          (reinterpret_cast<uintptr_t>(e.g) & (8 * sizeof(G) - 1)) |
                          ((reinterpret_cast<uintptr_t>(e.m) | reinterpret_cast<uintptr_t>(e.v)) & s_mask) |
                          (reinterpret_cast<uintptr_t>(e.copy) & 15u);
    e.vec = bad == 0u ? 1u : 0u;
    tab.first[i] = at;
    at += (e.numel + (uint32_t)kAwSeg - 1u) / (uint32_t)kAwSeg;
  }
  tab.first[count] = at;
  tab.count = count;
  tab.id0 = id0;
  tab.last = last ? 1 : 0;
  if (at == 0 && !last) return SBN_OK;
  const uint32_t grid = std::max(1u, std::min(at, (uint32_t)(cache[dev] * sms)));
  return launch_ex(kern, dim3(grid), dim3(kAwThreads), 0, st, 1, tab, hp);
}

template <typename P, typename G, int BITS>
sbn_status run_adamw(const sbn_adamw_tensor* t, int count, const AwHyper& hp, int sms, cudaStream_t st) {
  for (int at = 0; at < count; at += kAwLarge) {
    const int n = std::min(kAwLarge, count - at);
    const bool last = at + n == count;
    const sbn_status s = n <= kAwSmall
                             ? launch_adamw<P, G, BITS, kAwSmall>(t + at, n, (uint32_t)at, last, hp, sms, st)
                             : launch_adamw<P, G, BITS, kAwLarge>(t + at, n, (uint32_t)at, last, hp, sms, st);
    if (s != SBN_OK) return s;
  }
  return SBN_OK;
}

bool off_by(const void* p, uintptr_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0u; }

}  // namespace
}  // namespace sbn

using namespace sbn;

extern "C" sbn_status sbn_adamw(const sbn_adamw_tensor* tensors, int32_t count, int32_t p_bf16, int32_t g_bf16,
                                int32_t state_bits, int32_t* step, double lr, const float* lr_dev, double beta1,
                                double beta2, double eps, double weight_decay, const float* grad_scale, uint32_t seed,
                                void* stream) {
  if (!tensors || !step) return SBN_ERR_NULL;
  if (count < 1 || (state_bits != 8 && state_bits != 32)) return SBN_ERR_SHAPE;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= FLT_MIN) || !std::isfinite(eps) ||
      !std::isfinite(lr) || !std::isfinite(weight_decay))
    return SBN_ERR_SHAPE;
  if (off_by(step, 4) || off_by(lr_dev, 4) || off_by(grad_scale, 4)) return SBN_ERR_ALIGN;
  const uintptr_t ps = p_bf16 ? 2 : 4, gsz = g_bf16 ? 2 : 4, ss = state_bits == 32 ? 4 : 1;
  for (int32_t i = 0; i < count; ++i) {
    const sbn_adamw_tensor& t = tensors[i];
    if (t.numel < 0 || t.numel >= (1ll << 31)) return SBN_ERR_SHAPE;
    if (t.numel == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale))) return SBN_ERR_NULL;
    if (p_bf16 && t.copy_bf16) return SBN_ERR_SHAPE;
    if (off_by(t.p, ps) || off_by(t.g, gsz) || off_by(t.m, ss) || off_by(t.v, ss) || off_by(t.m_scale, 4) ||
        off_by(t.v_scale, 4) || off_by(t.copy_bf16, 2))
      return SBN_ERR_ALIGN;
  }
  int dev = 0, sms = 0;
  const sbn_status st = check_device(&dev, &sms);
  if (st != SBN_OK) return st;
  AwHyper hp;
  hp.step = step; hp.lr_dev = lr_dev; hp.gscale = grad_scale;
  hp.lr = lr; hp.wd = weight_decay; hp.log_b1 = std::log(beta1); hp.log_b2 = std::log(beta2);
  hp.b1 = (float)beta1; hp.omb1 = (float)(1.0 - beta1); hp.b2 = (float)beta2; hp.omb2 = (float)(1.0 - beta2);
  hp.eps = (float)eps;
  hp.seed = seed;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (state_bits == 32) {
    if (p_bf16) return g_bf16 ? run_adamw<uint16_t, uint16_t, 32>(tensors, count, hp, sms, cs)
                              : run_adamw<uint16_t, float, 32>(tensors, count, hp, sms, cs);
    return g_bf16 ? run_adamw<float, uint16_t, 32>(tensors, count, hp, sms, cs)
                  : run_adamw<float, float, 32>(tensors, count, hp, sms, cs);
  }
  if (p_bf16) return g_bf16 ? run_adamw<uint16_t, uint16_t, 8>(tensors, count, hp, sms, cs)
                            : run_adamw<uint16_t, float, 8>(tensors, count, hp, sms, cs);
  return g_bf16 ? run_adamw<float, uint16_t, 8>(tensors, count, hp, sms, cs)
                : run_adamw<float, float, 8>(tensors, count, hp, sms, cs);
}
