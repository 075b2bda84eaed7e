// Backward of the grouped layer: dX and dW of every expert's rows.
//
// "Microsoft BitNet 1.58: The Era of 1-Bit Large Language Models", section
// "Training with the Straight-Through Estimator", as in bwd_tc.cuh, per
// expert e with the rows r in its range:
//     dX_r = dY_r (gamma_e C_e)                  contraction over N_out
//     dW_e = sum_r dY_r^T (Xq_r s_r / 127)       contraction over e's rows
// on `tcgen05.mma.cta_group::1.kind::f16` with bf16 operands and fp32
// accumulation in tensor memory; an expert without rows has dW_e = 0, rows
// outside the experts' ranges keep their dX.
//
// dX: persistent CTAs walk tiles of 128 rows of one expert x 256 positions.
//   warp 0      TMA of dY (128 rows x 64 features per stage, K-major);
//   warp 1      TMEM and the MMA thread;  warp 2  the work list;
//   warps 4-11  producers: a thread expands 64 positions of one output
//               feature of C_e (bl_gemv.cuh's expansion) to bf16, one
//               128-byte row of the MN-major B tile;
//   warps 12-15 epilogue.
// Rows of the next expert in a tile are multiplied too (rows are
// independent) and not stored.
//
// dW: tiles of 128 features x 256 positions of one expert, 64 rows per
// stage. Xq is exact in bf16; a = fp32(dY s / 127) is split into a_hi =
// bf16(a) and a_lo = bf16(a - a_hi) (|a - a_hi - a_lo| <= 2^-18 |a|), two MMAs
// per step. Producers write all operands (MN-major), zeros behind the range.
#pragma once

#include <cuda.h>

#include "async.cuh"
#include "bl_gemv.cuh"
#include "bl_tc.cuh"
#include "bl_tc_grp.cuh"
#include "bwd.cuh"
#include "bwd_tc.cuh"
#include "common.cuh"
#include "grp.cuh"

namespace sbn {

constexpr int kGxSelCopies = kTgSelCopies;

__host__ __device__ inline size_t gx_smem_bytes(int experts) {
  return 1024 + (size_t)kBxStages * kBxStageBytes + 256 * 8 * kGxSelCopies + (2 * kBxStages + 4) * 8 + 16 +
         2 * 4 * (size_t)(experts + 1);
}
__host__ __device__ inline size_t gw_smem_bytes(int experts) {
  return kBwSmemBytes + 2 * 4 * (size_t)(experts + 1);
}

struct GxParams {
  const uint8_t* codes;
  const uint8_t* meta;
  const float* gamma;
  uint16_t* dx;
  GrpParams grp;
  int K, N;
  int cstride, mstride;
};

template <int MM, int CB, bool DENSE>
__global__ void __launch_bounds__(kTcThreads, 1)
bwd_dx_grp_kernel(const __grid_constant__ CUtensorMap tmap_dy, const GxParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint2* s_sel = reinterpret_cast<uint2*>(smem + (size_t)kBxStages * kBxStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(s_sel + 256 * kGxSelCopies);
  uint64_t* empty = full + kBxStages;
  uint64_t* acc_full = empty + kBxStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 4);
  int* s_first = s_off + p.grp.experts + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nst = (p.N + kBxBK - 1) / kBxBK;
  const int col_tiles = (p.K + kBxBN - 1) / kBxBN;

  if (tid == 0) {
    for (int s = 0; s < kBxStages; ++s) {
      mbar_init(&full[s], kTcProducers / 32 + 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kTcEpilogue / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(s_tmem)),
                 "r"(kBxTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (!DENSE) {
    for (int i = tid; i < 256 * kGxSelCopies; i += blockDim.x) s_sel[i] = gv_selector_pair((uint32_t)(i / kGxSelCopies));
  }
  griddep_wait();
  if (warp == 2) grp_build(p.grp, kBxBM, col_tiles, 0, s_off, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int n_tiles = s_first[p.grp.experts], grid = (int)gridDim.x;
  int used = 0;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
        const TgTile t = tg_tile(s_off, s_first, p.grp, tile, col_tiles, kBxBN, kBxBM, 1);
        if (!t.nmma) continue;
        for (int ks = 0; ks < nst; ++ks, ++it) {
          const int s = it % kBxStages;
          if (!mbar_wait(&empty[s], ((it / kBxStages) & 1u) ^ 1u)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[s], kBxABytes);
          tma_load_2d(smem + (size_t)s * kBxStageBytes, &tmap_dy, ks * kBxBK, t.tok0, &full[s]);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
        const TgTile t = tg_tile(s_off, s_first, p.grp, tile, col_tiles, kBxBN, kBxBM, 1);
        if (!t.nmma) continue;
        const int b = used & 1;
        if (!mbar_wait(&acc_empty[b], ((used >> 1) & 1u) ^ 1u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(b * kBxBN);
        for (int ks = 0; ks < nst; ++ks, ++it) {
          const int s = it % kBxStages;
          if (!mbar_wait(&full[s], (it / kBxStages) & 1u)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + (size_t)s * kBxStageBytes);
          const uint64_t adesc = sw128_kmajor_desc(a_addr);
          const uint64_t bdesc = sw128_mnmajor_desc(a_addr + kBxABytes, 1024u, 4096u);
#pragma unroll
          for (int k = 0; k < kBxBK / 16; ++k)
            tc_mma_f16(d_tmem, adesc + (uint64_t)(2 * k), bdesc + (uint64_t)(k * (8192 / 16)),
                       (ks > 0 || k > 0) ? 1u : 0u);
          tc_commit(&empty[s]);
        }
        tc_commit(&acc_full[b]);
        ++used;
      }
      for (int j = used - 2; j < used; ++j)
        if (j >= 0) mbar_wait(&acc_full[j & 1], (j >> 1) & 1u);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ---- producers: thread (feature ol of the stage, span q of 64 positions) ----
    const int pi = tid - 128, ol = pi & 63, q = pi >> 6;
    const uint2* sel = s_sel + (lane & (kGxSelCopies - 1));
    const int r = ol & 7;
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
      const TgTile t = tg_tile(s_off, s_first, p.grp, tile, col_tiles, kBxBN, kBxBM, 1);
      if (!t.nmma) continue;
      const int k0 = t.row0 + 64 * q;   // first position of the span
      const bool in_k = k0 < p.K;
      const uint8_t* crow = p.codes + (size_t)t.e * p.N * p.cstride + (size_t)(k0 >> 4) * CB;
      const uint8_t* mrow = DENSE ? nullptr : p.meta + (size_t)t.e * p.N * p.mstride + (k0 >> 3);
      uint32_t cn[CB], mn[2];
      auto load = [&](int ks) {
        const int o = ks * kBxBK + ol;
#pragma unroll
        for (int j = 0; j < CB; ++j) cn[j] = 0u;
        mn[0] = mn[1] = 0u;
        if (o < p.N && in_k) {
          const uint32_t* cp = reinterpret_cast<const uint32_t*>(crow + (size_t)o * p.cstride);
#pragma unroll
          for (int j = 0; j < CB; ++j) cn[j] = __ldg(cp + j);
          if (!DENSE) {
            const uint2 m = __ldg(reinterpret_cast<const uint2*>(mrow + (size_t)o * p.mstride));
            mn[0] = m.x;
            mn[1] = m.y;
          }
        }
      };
      load(0);
      for (int ks = 0; ks < nst; ++ks, ++it) {
        const int s = it % kBxStages;
        uint32_t cw[CB], mw[2] = {mn[0], mn[1]};
#pragma unroll
        for (int j = 0; j < CB; ++j) cw[j] = cn[j];
        if (ks + 1 < nst) load(ks + 1);
        uint32_t w[16];
        tg_expand64<MM, CB, DENSE>(cw, mw, sel, w);
        int got = 1;
        if (lane == 0) got = mbar_wait(&empty[s], ((it / kBxStages) & 1u) ^ 1u) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) { ok = false; break; }
        uint8_t* row = smem + (size_t)s * kBxStageBytes + kBxABytes + (size_t)(ol >> 3) * 4096 + (size_t)q * 1024 +
                       (size_t)r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t h[4];
          s8x4_to_bf16x4(w[2 * c], h[0], h[1]);
          s8x4_to_bf16x4(w[2 * c + 1], h[2], h[3]);
          *reinterpret_cast<uint4*>(row + ((c ^ r) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
  } else if (warp >= 12) {
    const int q = warp & 3;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    for (int tile = blockIdx.x; tile < n_tiles; tile += grid) {
      const TgTile t = tg_tile(s_off, s_first, p.grp, tile, col_tiles, kBxBN, kBxBM, 1);
      if (!t.nmma) continue;
      const int b = used & 1;
      const int row = t.tok0 + 32 * q + lane;
      const float g = __ldg(p.gamma + t.e);
      int got = 1;
      if (lane == 0) got = mbar_wait(&acc_full[b], (used >> 1) & 1u) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      ++used;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kBxBN / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(tmem + lane_base + (uint32_t)(b * kBxBN + 32 * c), r);
        const int kc = t.row0 + 32 * c;
        if (row < t.tok_end && kc < p.K) {
          uint32_t o16[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o16[e] = (uint32_t)f32_to_bf16_bits(__fmul_rn(g, __uint_as_float(r[2 * e]))) |
                     ((uint32_t)f32_to_bf16_bits(__fmul_rn(g, __uint_as_float(r[2 * e + 1]))) << 16);
          uint4* dst = reinterpret_cast<uint4*>(p.dx + (size_t)row * p.K + kc);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_uint4(o16[4 * e], o16[4 * e + 1], o16[4 * e + 2], o16[4 * e + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
    griddep_launch_dependents();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kBxTmemCols) : "memory");
  }
}

struct GwParams {
  const uint16_t* dy;
  const int8_t* xq;
  const float* xs;
  uint16_t* dw;     // [E, N, K]
  GrpParams grp;
  int K, N;
};

static __global__ void __launch_bounds__(kTcThreads, 1) bwd_dw_grp_kernel(const GwParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)kBwStages * kBwStageBytes);
  uint64_t* empty = full + kBwStages;
  uint64_t* acc_full = empty + kBwStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 4);
  int* s_first = s_off + p.grp.experts + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int col_tiles = (p.K + kBwBN - 1) / kBwBN;
  const int per_expert = col_tiles * ((p.N + kBwBM - 1) / kBwBM);
  const int n_tiles = p.grp.experts * per_expert, grid = (int)gridDim.x;

  if (tid == 0) {
    for (int s = 0; s < kBwStages; ++s) {
      mbar_init(&full[s], kTcProducers / 32);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kTcEpilogue / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(s_tmem)),
                 "r"(kBxTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  griddep_wait();
  if (warp == 2) grp_build(p.grp, 1, 0, 0, s_off, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  int used = 0;

  if (warp == 1) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
        const int e = tile / per_expert;
        const int nst = (s_off[e + 1] - s_off[e] + kBwBK - 1) / kBwBK;
        if (nst == 0) continue;
        const int b = used & 1;
        if (!mbar_wait(&acc_empty[b], ((used >> 1) & 1u) ^ 1u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(b * kBwBN);
        for (int ks = 0; ks < nst; ++ks, ++it) {
          const int s = it % kBwStages;
          if (!mbar_wait(&full[s], (it / kBwStages) & 1u)) { ok = false; break; }
          tc_fence_after();
          const uint32_t base = smem_u32(smem + (size_t)s * kBwStageBytes);
          const uint64_t ahi = sw128_mnmajor_desc(base, 1024u, 2048u);
          const uint64_t alo = sw128_mnmajor_desc(base + kBwAPlane, 1024u, 2048u);
          const uint64_t bd = sw128_mnmajor_desc(base + 2 * kBwAPlane, 1024u, 4096u);
#pragma unroll
          for (int k = 0; k < kBwBK / 16; ++k) {
            tc_mma_f16_mn(d_tmem, ahi + (uint64_t)(k * (4096 / 16)), bd + (uint64_t)(k * (8192 / 16)),
                          (ks > 0 || k > 0) ? 1u : 0u);
            tc_mma_f16_mn(d_tmem, alo + (uint64_t)(k * (4096 / 16)), bd + (uint64_t)(k * (8192 / 16)), 1u);
          }
          tc_commit(&empty[s]);
        }
        tc_commit(&acc_full[b]);
        ++used;
      }
      for (int j = used - 2; j < used; ++j)
        if (j >= 0) mbar_wait(&acc_full[j & 1], (j >> 1) & 1u);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    const int pi = tid - 128;
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
      const int e = tile / per_expert, local = tile - e * per_expert;
      const int lo = s_off[e], hi = s_off[e + 1];
      const int nst = (hi - lo + kBwBK - 1) / kBwBK;
      const int o0 = (local / col_tiles) * kBwBM, k0 = (local % col_tiles) * kBwBN;
      for (int ks = 0; ks < nst; ++ks, ++it) {
        const int s = it % kBwStages;
        int got = 1;
        if (lane == 0) got = mbar_wait(&empty[s], ((it / kBwStages) & 1u) ^ 1u) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) { ok = false; break; }
        uint8_t* st = smem + (size_t)s * kBwStageBytes;
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int i = pi + 256 * q4, tl = i >> 4, f8 = i & 15;
          const int t = lo + ks * kBwBK + tl, r = tl & 7;
          {   // A: row t, features 8 f8 ..
            const int o = o0 + 8 * f8;
            uint4 hi4 = make_uint4(0u, 0u, 0u, 0u), lo4 = hi4;
            if (t < hi && o < p.N) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.dy + (size_t)t * p.N + o));
              scale_split8(v, __fdiv_rn(__ldg(p.xs + t), 127.0f), hi4, lo4);
            }
            const size_t off = (size_t)(tl >> 3) * 2048 + (size_t)(f8 >> 3) * 1024 + (size_t)r * 128 + (((f8 & 7) ^ r) << 4);
            *reinterpret_cast<uint4*>(st + off) = hi4;
            *reinterpret_cast<uint4*>(st + kBwAPlane + off) = lo4;
          }
          {   // B: row t, positions 16 u ..
            const int u = f8, kk = k0 + 16 * u;
            uint32_t h[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            if (t < hi && kk < p.K) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.xq + (size_t)t * p.K + kk));
              s8x4_to_bf16x4_any(v.x, h[0], h[1]);
              s8x4_to_bf16x4_any(v.y, h[2], h[3]);
              s8x4_to_bf16x4_any(v.z, h[4], h[5]);
              s8x4_to_bf16x4_any(v.w, h[6], h[7]);
            }
            const int c0 = 2 * (u & 3);
            uint8_t* atom = st + 2 * kBwAPlane + (size_t)(tl >> 3) * 4096 + (size_t)(u >> 2) * 1024 + (size_t)r * 128;
            *reinterpret_cast<uint4*>(atom + ((c0 ^ r) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(atom + (((c0 + 1) ^ r) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
  } else if (warp >= 12) {
    const int q = warp & 3;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    for (int tile = blockIdx.x; tile < n_tiles; tile += grid) {
      const int e = tile / per_expert, local = tile - e * per_expert;
      const bool any = s_off[e + 1] > s_off[e];
      const int b = used & 1;
      const int o = (local / col_tiles) * kBwBM + 32 * q + lane, k0 = (local % col_tiles) * kBwBN;
      if (any) {
        int got = 1;
        if (lane == 0) got = mbar_wait(&acc_full[b], (used >> 1) & 1u) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) break;
        ++used;
        tc_fence_after();
      }
      uint16_t* drow = p.dw + ((size_t)e * p.N + o) * p.K;
#pragma unroll 1
      for (int c = 0; c < kBwBN / 32; ++c) {
        uint32_t r[32];
        if (any) {
          tmem_ld32(tmem + lane_base + (uint32_t)(b * kBwBN + 32 * c), r);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        const int kc = k0 + 32 * c;
        if (o < p.N && kc < p.K) {
          uint32_t o16[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o16[i] = (uint32_t)f32_to_bf16_bits(__uint_as_float(r[2 * i])) |
                     ((uint32_t)f32_to_bf16_bits(__uint_as_float(r[2 * i + 1])) << 16);
          uint4* dst = reinterpret_cast<uint4*>(drow + kc);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_uint4(o16[4 * i], o16[4 * i + 1], o16[4 * i + 2], o16[4 * i + 3]);
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[b]);
      }
    }
    griddep_launch_dependents();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kBxTmemCols) : "memory");
  }
}

// ---------------------------------------------------------------------------
// N_out not a multiple of 8 (dY's rows do not start on 16-byte boundaries):
// tiled fp32 products on the CUDA cores, as in bwd.cuh.
// ---------------------------------------------------------------------------
template <int MM, int CB, bool DENSE>
__global__ void __launch_bounds__(kBwThreads)
bwd_dx_grp_plain_kernel(const uint16_t* __restrict__ dy, const GxParams p) {
  extern __shared__ int s_list[];
  __shared__ float s_a[kBwSlice][kBwTile];   // dY^T slice: [n][t]
  __shared__ float s_b[kBwSlice][kBwTile];   // C slice: [n][k]
  int* s_off = s_list;
  int* s_first = s_list + p.grp.experts + 1;
  griddep_wait();
  if (threadIdx.x < 32) grp_build(p.grp, kBwTile, 1, 0, s_off, s_first);
  __syncthreads();
  if ((int)blockIdx.y >= s_first[p.grp.experts]) return;
  const TgTile tl = tg_tile(s_off, s_first, p.grp, blockIdx.y, 1, 0, kBwTile, 1);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int k0 = blockIdx.x * kBwTile;
  const uint8_t* codes = p.codes + (size_t)tl.e * p.N * p.cstride;
  const uint8_t* meta = DENSE ? nullptr : p.meta + (size_t)tl.e * p.N * p.mstride;
  float acc[4][4] = {};
  for (int n0 = 0; n0 < p.N; n0 += kBwSlice) {
    for (int i = tid; i < kBwSlice * kBwTile; i += kBwThreads) {
      const int tt = i / kBwSlice, nn = i - tt * kBwSlice;
      const int t = tl.tok0 + tt, n = n0 + nn;
      s_a[nn][tt] = (t < tl.tok_end && n < p.N) ? bf16_to_f32(dy[(size_t)t * p.N + n]) : 0.f;
    }
    if (tid < kBwSlice * (kBwTile / 16)) {
      const int nn = tid >> 2, uu = tid & 3;
      const int n = n0 + nn, u = (k0 >> 4) + uu;
      uint32_t cw = 0u, keep = 0u;
      if (n < p.N) {
        const uint8_t* cp = codes + (size_t)n * p.cstride + (size_t)u * CB;
#pragma unroll
        for (int b = 0; b < CB; ++b) cw |= (uint32_t)cp[b] << (8 * b);
        keep = DENSE ? 0xFFFFu
                     : (uint32_t)meta[(size_t)n * p.mstride + 2 * u] | ((uint32_t)meta[(size_t)n * p.mstride + 2 * u + 1] << 8);
      }
      int ci = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float v = 0.f;
        if ((keep >> j) & 1u) {
          const uint32_t c2 = (cw >> (2 * ci)) & 3u;
          v = (c2 == 1u) ? 1.f : ((c2 == 3u) ? -1.f : 0.f);
          ++ci;
        }
        s_b[nn][uu * 16 + j] = v;
      }
    }
    __syncthreads();
    bw_slice_fma(s_a, s_b, ty, tx, acc);
    __syncthreads();
  }
  const float g = __ldg(p.gamma + tl.e);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = tl.tok0 + ty * 4 + i;
    if (t >= tl.tok_end) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) p.dx[(size_t)t * p.K + k0 + tx * 4 + j] = f32_to_bf16_bits(__fmul_rn(g, acc[i][j]));
  }
}

// Grid (K / 64, ceil(N_out / 64), E).
static __global__ void __launch_bounds__(kBwThreads) bwd_dw_grp_plain_kernel(const GwParams p) {
  extern __shared__ int s_list[];
  __shared__ float s_a[kBwSlice][kBwTile];   // dY slice: [t][n]
  __shared__ float s_b[kBwSlice][kBwTile];   // Xd slice: [t][k]
  griddep_wait();
  if (threadIdx.x < 32) grp_build(p.grp, 1, 0, 0, s_list, s_list + p.grp.experts + 1);
  __syncthreads();
  const int e = (int)blockIdx.z, lo = s_list[e], hi = s_list[e + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int k0 = blockIdx.x * kBwTile, n0 = blockIdx.y * kBwTile;
  float acc[4][4] = {};
  for (int t0 = lo; t0 < hi; t0 += kBwSlice) {
    for (int i = tid; i < kBwSlice * kBwTile; i += kBwThreads) {
      const int tt = i / kBwTile, cc = i - tt * kBwTile;
      const int t = t0 + tt;
      const bool tok = t < hi;
      s_a[tt][cc] = (tok && n0 + cc < p.N) ? bf16_to_f32(p.dy[(size_t)t * p.N + n0 + cc]) : 0.f;
      s_b[tt][cc] = tok ? (float)p.xq[(size_t)t * p.K + k0 + cc] * __fdiv_rn(__ldg(p.xs + t), 127.0f) : 0.f;
    }
    __syncthreads();
    bw_slice_fma(s_a, s_b, ty, tx, acc);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + ty * 4 + i;
    if (n >= p.N) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      p.dw[((size_t)e * p.N + n) * p.K + k0 + tx * 4 + j] = f32_to_bf16_bits(acc[i][j]);
  }
}

}  // namespace sbn
