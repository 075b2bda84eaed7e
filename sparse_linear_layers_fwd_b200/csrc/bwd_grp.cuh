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
// dX: persistent CTAs walk tiles of 128 rows of one expert x 256 positions,
// 64 features of the contraction per stage.
//   warp 0      TMA of dY (128 rows x 64 features, K-major);
//   warp 1      TMEM and the MMA warp;
//   warp 2      the work list, then TMA of the packed rows (64 features x 256
//               positions of codes and keep bits);
//   warps 4-19  producers: two groups of eight warps take the stages in turn; a
//               thread expands 64 positions of one output feature of C_e
//               (bl_gemv.cuh's expansion) to bf16, one 128-byte row of the
//               MN-major B tile. The byte table gives the high byte of bf16
//               0, 1 or -1, whose low byte is its lowest bit moved up;
//   warps 20-23 epilogue.
// Rows of the next expert in a tile are multiplied too (rows are
// independent) and not stored. Bound by shared memory: a stage's MMAs read 48
// KB, TMA writes 16 and the producers 32, 768 cycles at 128 bytes each beside
// 512 cycles of MMA.
//
// dW in two kernels. bwd_dw_prep_kernel lays the operands out once in the
// caller's workspace, as fp16, every expert's rows padded with zeros to a
// multiple of 64: Xq (exact) and a = dY s / 127 times a power of two per
// (expert, feature) that brings the largest |a| of the feature just below
// 2^15. a is held in two fp16 parts, a rounded and what that leaves: together 22
// bits of it, or 2^-39 of the feature's largest. With one part (11 bits; a
// workspace of that size) the MMAs are halved: 152 us in place of 189 for dX and dW
// at 8192 rows, and the error after the rounding of dW to bf16 is the same to
// 1 % (1.67e-3 against 1.66e-3) - but not where terms cancel: rows in pairs of
// opposite gradients and nearly the same activations leave 1.5e-2, two parts
// 1.66e-3, the two bf16 parts of bwd_tc.cuh 1.67e-3. bwd_dw_grp_kernel then is a
// plain TMA-fed product over tiles of 128 features x 256 positions, two MMAs for
// every 16 rows into the same accumulator, both operands MN-major (features and
// positions are contiguous in a row): 1 KB atoms of 8 rows x 64 columns.
// Converting in the product's own producer warps instead, for every tile
// again, took six times as long as its MMAs.
// Its tiles leave through shared memory and TMA stores: from registers, each
// lane writing its feature's 64 bytes, it took 57 us in place of 48 (one part).
//
// Where N_out is not a multiple of 8, dY's rows do not start on 16-byte
// boundaries: dW's preparation reads them two bytes at a time, and dX gets a
// copy of dY at a padded pitch first (bwd_pitch_kernel).
// Measured launch by launch on cold caches at 8192 rows of 16 experts (K = 2048,
// N_out = 1408, 6:8): dX 72 us, preparation 51 (one part 43), dW 73 (0.76 of the
// bf16 rate; one part 50); at 1000 rows (K = 896, N_out = 1000, 8:16) 20, 13 and
// 17.5 us (dW of one part 16.5). Back to back they overlap: 189 and 40 us in all.
#pragma once

#include <cuda.h>

#include "async.cuh"
#include "bl_gemv.cuh"
#include "bl_tc.cuh"
#include "bl_tc_grp.cuh"
#include "bwd_tc.cuh"
#include "common.cuh"
#include "grp.cuh"

namespace sbn {

constexpr int kGxSelCopies = 4;
constexpr int kGxThreads = 768;
constexpr int kGxEpiWarp = 20;                       // first epilogue warp
constexpr int kGxPackedBytes = kBxBK * (48 + 32);    // packed rows of a stage, at most (6:8)
constexpr int kGxPacked = 4;                         // their ring; even, so that a slot stays with one group and
                                                     // its parity waits never span two rounds
constexpr int kGxList = 32;
constexpr uint32_t kBf16HighTable = 0xBF003F00u;     // codes 00, 01, 10, 11 -> high byte of bf16

__host__ __device__ inline size_t gx_smem_bytes(int experts) {
  return 1024 + (size_t)kBxStages * kBxStageBytes + kGxPacked * kGxPackedBytes + 256 * 4 * kGxSelCopies +
         (2 * (kBxStages + kGxPacked) + 4) * 8 + 16 + 16 * kGxList + 2 * 4 * (size_t)(experts + 1);
}

// Eight positions (group I of the span) -> eight bf16 (0, 1 or -1).
template <int MM, int CB, bool DENSE, int I>
SBN_DEVFN uint4 gx_expand8(const uint32_t (&cw)[CB], const uint32_t (&mw)[2], const uint32_t* sel) {
  uint32_t h0, h1;
  gv_expand<MM, CB, DENSE, I, kGxSelCopies, kBf16HighTable>(cw, mw, sel, h0, h1);
  const uint32_t l0 = (h0 << 7) & 0x80808080u, l1 = (h1 << 7) & 0x80808080u;
  return make_uint4(gv_prmt(l0, h0, 0x5140u), gv_prmt(l0, h0, 0x7362u), gv_prmt(l1, h1, 0x5140u),
                    gv_prmt(l1, h1, 0x7362u));
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
__global__ void __launch_bounds__(kGxThreads, 1)
bwd_dx_grp_kernel(const __grid_constant__ CUtensorMap tmap_dy, const __grid_constant__ CUtensorMap tmap_c,
                  const __grid_constant__ CUtensorMap tmap_m, const GxParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* packed = smem + (size_t)kBxStages * kBxStageBytes;
  uint32_t* s_sel = reinterpret_cast<uint32_t*>(packed + kGxPacked * kGxPackedBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(s_sel + 256 * kGxSelCopies);
  uint64_t* empty = full + kBxStages;
  uint64_t* p_full = empty + kBxStages;
  uint64_t* p_empty = p_full + kGxPacked;
  uint64_t* acc_full = p_empty + kGxPacked;   // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int4* s_list = reinterpret_cast<int4*>(s_tmem + 4);
  int* s_off = reinterpret_cast<int*>(s_list + kGxList);
  int* s_first = s_off + p.grp.experts + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nst = (p.N + kBxBK - 1) / kBxBK;
  const int col_tiles = (p.K + kBxBN - 1) / kBxBN;

  if (tid == 0) {
    for (int s = 0; s < kBxStages; ++s) {
      mbar_init(&full[s], 8 + 1);   // a group's warps and dY's TMA
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kGxPacked; ++s) {
      mbar_init(&p_full[s], 1);
      mbar_init(&p_empty[s], 8);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
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
    for (int i = tid; i < 256 * kGxSelCopies; i += blockDim.x) s_sel[i] = gv_selector((uint32_t)(i / kGxSelCopies));
  }
  griddep_wait();
  if (warp == 2) grp_build(p.grp, kBxBM, col_tiles, 0, s_off, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int n_tiles = s_first[p.grp.experts];
  const int count = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  tg_list<kBxBN, kBxBM, 1>(s_list, kGxList, s_off, s_first, p.grp, count, col_tiles);
  __syncthreads();
  auto tile_at = [&](int k) { return tg_get<kBxBN, kBxBM, 1>(s_list, kGxList, s_off, s_first, p.grp, k, col_tiles); };
  int used = 0;

  if (warp == 0) {
    const bool lead = elect_one();
    int s = 0;
    uint32_t ph = 1u;
    bool ok = true;
    for (int k = 0; k < count && ok; ++k) {
      const TgTile t = tile_at(k);
      if (!t.nmma) continue;
      const int tok0 = __shfl_sync(0xffffffffu, t.tok0, 0);
      for (int ks = 0; ks < nst; ++ks) {
        if (!mbar_wait_warp(&empty[s], ph)) { ok = false; break; }
        uint8_t* st = smem + (size_t)s * kBxStageBytes;
        if (lead) {
          mbar_arrive_expect_tx(&full[s], kBxABytes);
          tma_load_2d(st, &tmap_dy, ks * kBxBK, tok0, &full[s]);
        }
        __syncwarp();
        if (++s == kBxStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 2) {
    const bool lead = elect_one();
    int it = 0;
    bool ok = true;
    for (int k = 0; k < count && ok; ++k) {
      const TgTile t = tile_at(k);
      if (!t.nmma) continue;
      // rows past the expert's (of the next, or zeros) meet zeros of dY
      const int row = __shfl_sync(0xffffffffu, t.e * p.N, 0), k0 = __shfl_sync(0xffffffffu, t.row0, 0);
      for (int ks = 0; ks < nst; ++ks, ++it) {
        const int s = it % kGxPacked;
        if (!mbar_wait_warp(&p_empty[s], ((it / kGxPacked) & 1u) ^ 1u)) { ok = false; break; }
        uint8_t* dst = packed + s * kGxPackedBytes;
        if (lead) {
          mbar_arrive_expect_tx(&p_full[s], (uint32_t)(kBxBK * (16 * CB + (DENSE ? 0 : 32))));
          tma_load_2d(dst, &tmap_c, k0 / 16 * CB, row + ks * kBxBK, &p_full[s]);
          if (!DENSE) tma_load_2d(dst + kBxBK * 16 * CB, &tmap_m, k0 / 8, row + ks * kBxBK, &p_full[s]);
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer: the whole warp runs the loop, one elected lane issues ----
    const bool lead = elect_one();
    const uint32_t base = smem_u32(smem);
    const uint64_t ad0 = sw128_kmajor_desc(base), bd0 = sw128_mnmajor_desc(base + kBxABytes, 1024u, 4096u);
    int s = 0;
    uint32_t ph = 0u;
    bool ok = true;
    for (int k = 0; k < count && ok; ++k) {
      const TgTile t = tile_at(k);
      if (!t.nmma) continue;
      const int b = used & 1;
      if (!mbar_wait_warp(&acc_empty[b], ((used >> 1) & 1u) ^ 1u)) break;
      const uint32_t d_tmem = tmem + (uint32_t)(b * kBxBN);
      for (int ks = 0; ks < nst; ++ks) {
        if (!mbar_wait_warp(&full[s], ph)) { ok = false; break; }
        tc_fence_after();
        const uint64_t so = (uint64_t)(s * (kBxStageBytes / 16));
        if (lead) {
#pragma unroll
          for (int i = 0; i < kBxBK / 16; ++i)
            tc_mma_f16(d_tmem, ad0 + so + (uint64_t)(2 * i), bd0 + so + (uint64_t)(i * (8192 / 16)),
                       (ks > 0 || i > 0) ? 1u : 0u);
          tc_commit(&empty[s]);
        }
        __syncwarp();
        if (++s == kBxStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (lead) tc_commit(&acc_full[b]);
      __syncwarp();
      ++used;
    }
    for (int j = used - 2; j < used; ++j)
      if (j >= 0) mbar_wait(&acc_full[j & 1], (j >> 1) & 1u);
    __syncwarp();
  } else if (warp >= 4 && warp < kGxEpiWarp) {
    // ---- producers: group g takes the stages with index = g (mod 2), counted
    // over all tiles; thread = (feature ol of the stage, span q of 64 positions) ----
    const int g = (warp - 4) >> 3, pi = tid - 128 - 256 * g, ol = pi & 63, q = pi >> 6;
    const uint32_t* sel = s_sel + (lane & (kGxSelCopies - 1));
    const int r = ol & 7;
    uint8_t* const row0 = smem + kBxABytes + (size_t)(ol >> 3) * 4096 + (size_t)q * 1024 + (size_t)r * 128;
    int it = 0;
    bool ok = true;
    for (int k = 0; k < count && ok; ++k) {
      const TgTile t = tile_at(k);
      if (!t.nmma) continue;
      const int end = it + nst;
      int mine = it + ((it ^ g) & 1);
      it = end;
      for (; mine < end; mine += 2) {
        const int ps = mine % kGxPacked;
        if (!mbar_wait_warp(&p_full[ps], (mine / kGxPacked) & 1u)) { ok = false; break; }
        const uint32_t* cp = reinterpret_cast<const uint32_t*>(packed + ps * kGxPackedBytes + ol * 16 * CB + q * 4 * CB);
        const uint2* mp = reinterpret_cast<const uint2*>(packed + ps * kGxPackedBytes + kBxBK * 16 * CB + ol * 32 + q * 8);
        uint32_t cw[CB], mw[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < CB; ++j) cw[j] = cp[j];
        if (!DENSE) {
          const uint2 m = *mp;
          mw[0] = m.x;
          mw[1] = m.y;
        }
        const int s = mine % kBxStages;
        if (!mbar_wait_warp(&empty[s], ((mine / kBxStages) & 1u) ^ 1u)) { ok = false; break; }
        uint8_t* row = row0 + (size_t)s * kBxStageBytes;
        *reinterpret_cast<uint4*>(row + ((0 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 0>(cw, mw, sel);
        *reinterpret_cast<uint4*>(row + ((1 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 1>(cw, mw, sel);
        *reinterpret_cast<uint4*>(row + ((2 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 2>(cw, mw, sel);
        *reinterpret_cast<uint4*>(row + ((3 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 3>(cw, mw, sel);
        *reinterpret_cast<uint4*>(row + ((4 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 4>(cw, mw, sel);
        *reinterpret_cast<uint4*>(row + ((5 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 5>(cw, mw, sel);
        *reinterpret_cast<uint4*>(row + ((6 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 6>(cw, mw, sel);
        *reinterpret_cast<uint4*>(row + ((7 ^ r) << 4)) = gx_expand8<MM, CB, DENSE, 7>(cw, mw, sel);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          // only now: handed back right behind the loads above, the packed rows
          // were overwritten before every lane's loads had been done
          mbar_arrive(&p_empty[ps]);
          mbar_arrive(&full[s]);
        }
      }
    }
  } else if (warp >= kGxEpiWarp) {
    const int q = warp & 3;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    for (int k = 0; k < count; ++k) {
      const TgTile t = tile_at(k);
      if (!t.nmma) continue;
      const int b = used & 1;
      const int row = t.tok0 + 32 * q + lane;
      const float gm = __ldg(p.gamma + t.e);
      if (!mbar_wait_warp(&acc_full[b], (used >> 1) & 1u)) break;
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
            o16[e] = (uint32_t)f32_to_bf16_bits(__fmul_rn(gm, __uint_as_float(r[2 * e]))) |
                     ((uint32_t)f32_to_bf16_bits(__fmul_rn(gm, __uint_as_float(r[2 * e + 1]))) << 16);
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

// Eight columns of a row of dY; WHOLE: its rows start on 16-byte boundaries
// (N_out a multiple of 8), otherwise columns past the last are zeros.
template <bool WHOLE>
SBN_DEVFN uint4 gw_load8(const uint16_t* dy, size_t row, int N, int col) {
  if constexpr (WHOLE) {
    return __ldg(reinterpret_cast<const uint4*>(dy + row * N + col));
  } else {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = col + i < N ? __ldg(dy + row * N + col + i) : 0u;
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
  }
}

// dY for dX where N_out is not a multiple of 8: rows copied to a pitch of
// round_up(N_out, 8), which TMA can load. Bound by DRAM and L2, 4 bytes per
// element; the alternative, 2-byte loads in the product's own warps, would repeat
// them for every 256 positions of K.
constexpr int kGcThreads = 256;
static __global__ void __launch_bounds__(kGcThreads)
bwd_pitch_kernel(const uint16_t* __restrict__ dy, uint16_t* __restrict__ dst, int rows, int N) {
  griddep_wait();
  const int per_row = (N + 7) / 8;
  const long long n = (long long)rows * per_row;
  for (long long i = (long long)blockIdx.x * kGcThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kGcThreads) {
    const long long row = i / per_row;
    const int c = (int)(i - row * per_row);
    reinterpret_cast<uint4*>(dst)[i] = gw_load8<false>(dy, (size_t)row, N, 8 * c);
  }
  griddep_launch_dependents();
}

struct GwParams {
  const uint16_t* dy;
  const int8_t* xq;
  const float* xs;
  uint16_t* dw;     // [E, N, K]
  GrpParams grp;
  int K, N;
  int Np;           // N rounded up to a multiple of 8
  // workspace: fp16 [padded rows, Np] and [padded rows, K], and the factor
  // that undoes the scaling of a, [E, N]
  uint16_t* a16;
  uint16_t* x16;
  float* scale;
  long long a_rows; // two parts of a: the padded rows of the first, the second follows; one part: 0
  int cluster;      // CTAs per (expert, 64 columns) in the preparation
  int a_ctas;       // its CTAs that scale dY; the others convert Xq
};

// Rows of the padded operands: every expert with rows ends a block of 64.
__host__ __device__ inline long long gw_padded_rows(int rows, int experts) {
  return ((long long)rows + 63ll * (experts < rows ? experts : rows)) / 64 * 64;
}

constexpr int kGpThreads = 256;
constexpr int kGpCols = 64;
constexpr int kGpLanes = kGpThreads / 8;   // row lanes: 8 threads x 8 columns make a row of 64

// CTAs [0, a_ctas): cluster c of (expert, column block), blockIdx = ((expert *
// blocks) + block) * cluster + rank: the features' largest |a| over the
// expert's rows, then a scaled. The other CTAs: Xq to fp16, one row (of a
// block of 64) per warp.
template <bool WHOLE>
__global__ void __launch_bounds__(kGpThreads) bwd_dw_prep_kernel(const GwParams p) {
  extern __shared__ int s_list[];
  __shared__ uint32_t s_max[kGpCols];
  __shared__ float s_mult[kGpCols];
  int* s_off = s_list;
  int* s_first = s_list + p.grp.experts + 1;   // blocks of 64 rows before an expert
  const int tid = threadIdx.x;
  griddep_wait();
  if (tid < 32) grp_build(p.grp, 64, 1, 0, s_off, s_first);
  if (tid < kGpCols) s_max[tid] = 0u;
  __syncthreads();
  const int blocks = (p.N + kGpCols - 1) / kGpCols;
  if ((int)blockIdx.x < p.a_ctas) {
    const int rank = (int)blockIdx.x % p.cluster, eb = (int)blockIdx.x / p.cluster;
    const int e = eb / blocks, c0 = (eb - e * blocks) * kGpCols;
    const int lo = s_off[e], hi = s_off[e + 1];
    const int col = c0 + 8 * (tid & 7), lane_r = tid >> 3;
    const bool in = col < p.Np;
    const int step = p.cluster * kGpLanes;
    uint32_t top[8] = {};
    for (int r0 = lo + rank * kGpLanes + lane_r; r0 < hi; r0 += 4 * step) {
      uint4 v[4];
      float sc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + u * step;
        const bool ok = in && r < hi;
        v[u] = ok ? gw_load8<WHOLE>(p.dy, (size_t)r, p.N, col) : make_uint4(0u, 0u, 0u, 0u);
        sc[u] = ok ? __fdiv_rn(__ldg(p.xs + r), 127.0f) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          top[2 * j] = max(top[2 * j], __float_as_uint(fabsf(__fmul_rn(__uint_as_float(w[j] << 16), sc[u]))));
          top[2 * j + 1] = max(top[2 * j + 1], __float_as_uint(fabsf(__fmul_rn(__uint_as_float(w[j] & 0xFFFF0000u), sc[u]))));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // lanes 8 apart share the columns
      top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
      top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
      if ((tid & 31) < 8) atomicMax(&s_max[8 * (tid & 7) + j], top[j]);
    }
    __syncthreads();
    if (p.cluster > 1) cluster_sync_all();
    if (tid < kGpCols) {
      uint32_t m = s_max[tid];
      for (int c = 0; c < p.cluster; ++c) {
        if (c == rank) continue;
        uint32_t o;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(o) : "r"(map_to_rank(smem_u32(&s_max[tid]), (uint32_t)c)));
        m = max(m, o);
      }
      const int ex = min(max((int)(m >> 23) - 127, -100), 126);
      s_mult[tid] = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
      if (rank == 0 && c0 + tid < p.N)
        p.scale[(size_t)e * p.N + c0 + tid] = __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
    }
    if (p.cluster > 1) cluster_sync_all();   // no CTA leaves while its maxima are read
    __syncthreads();
    const int pad_hi = lo + (hi - lo + 63) / 64 * 64;
    uint16_t* dst = p.a16 + ((size_t)s_first[e] * 64) * p.Np + col;
    float mult[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) mult[j] = s_mult[8 * (tid & 7) + j];
    for (int r0 = lo + rank * kGpLanes + lane_r; r0 < pad_hi; r0 += 4 * step) {
      uint4 v[4];
      float sc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + u * step;
        const bool ok = in && r < hi;
        v[u] = ok ? gw_load8<WHOLE>(p.dy, (size_t)r, p.N, col) : make_uint4(0u, 0u, 0u, 0u);
        sc[u] = ok ? __fdiv_rn(__ldg(p.xs + r), 127.0f) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + u * step;
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t h[4], l[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a0 = __fmul_rn(__fmul_rn(__uint_as_float(w[j] << 16), sc[u]), mult[2 * j]);
          const float a1 = __fmul_rn(__fmul_rn(__uint_as_float(w[j] & 0xFFFF0000u), sc[u]), mult[2 * j + 1]);
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(a1), "f"(a0));
          if (!p.a_rows) continue;
          // what the first part leaves, exact in fp32
          float h0, h1;
          asm("{\n.reg .f16 x, y;\nmov.b32 {x, y}, %2;\ncvt.f32.f16 %0, x;\ncvt.f32.f16 %1, y;\n}\n" : "=f"(h0), "=f"(h1) : "r"(h[j]));
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(l[j]) : "f"(__fsub_rn(a1, h1)), "f"(__fsub_rn(a0, h0)));
        }
        if (in && r < pad_hi) {
          uint16_t* at = dst + (size_t)(r - lo) * p.Np;
          *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
          if (p.a_rows) *reinterpret_cast<uint4*>(at + (size_t)p.a_rows * p.Np) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
    }
    griddep_launch_dependents();
    return;
  }
  // ---- Xq: warp w of these CTAs takes padded rows w, w + warps, ... ----
  const int n_rows = s_first[p.grp.experts] * 64;
  const int warps = ((int)gridDim.x - p.a_ctas) * (kGpThreads / 32);
  const int lane = tid & 31;
  for (int pr = ((int)blockIdx.x - p.a_ctas) * (kGpThreads / 32) + (tid >> 5); pr < n_rows; pr += warps) {
    const int e = grp_find(s_first, p.grp.experts, pr >> 6);
    const int r = s_off[e] + pr - s_first[e] * 64;
    const bool ok = r < s_off[e + 1];
    const uint4* src = reinterpret_cast<const uint4*>(p.xq + (size_t)r * p.K);
    uint4* d = reinterpret_cast<uint4*>(p.x16 + (size_t)pr * p.K);
    for (int c0 = lane; c0 < p.K / 16; c0 += 128) {
      uint4 vv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        vv[u] = ok && c0 + 32 * u < p.K / 16 ? __ldg(src + c0 + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
      const int c = c0 + 32 * u;
      if (c >= p.K / 16) break;
      uint32_t h[8];
      const uint32_t w[4] = {vv[u].x, vv[u].y, vv[u].z, vv[u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // bytes b + 128 as the low mantissa bits of 1024: exact, then - 1152
        const uint32_t u = w[j] ^ 0x80808080u;
        const uint32_t lo2 = __byte_perm(u, 0x64646464u, 0x4140u), hi2 = __byte_perm(u, 0x64646464u, 0x4342u);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * j]) : "r"(lo2), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * j + 1]) : "r"(hi2), "r"(0x64806480u));
      }
      d[2 * c] = make_uint4(h[0], h[1], h[2], h[3]);
      d[2 * c + 1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
    }
  }
  griddep_launch_dependents();
}

constexpr int kGwBM = 128;                       // features per tile (MMA M)
constexpr int kGwBN = 256;                       // positions per tile (MMA N)
constexpr int kGwBK = 64;                        // rows per stage
constexpr int kGwPart = kGwBM * kGwBK * 2;       // a part of a in a stage, 16 KB
constexpr int kGwRing = 192 * 1024;              // three stages of two parts, four of one
constexpr int kGwMaxStages = 4;
constexpr int kGwThreads = 384;                  // TMA, MMA, list, -, eight epilogue warps
constexpr int kGwOut = 8 * 2048;                 // a warp's 32 features x 32 positions of dW
// instruction descriptor: f32 accumulate, fp16 A and B, both MN-major
constexpr uint32_t kGwIdesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(kGwBN >> 3) << 17) |
                              ((uint32_t)(kGwBM >> 4) << 24);

__host__ __device__ inline size_t gw_smem_bytes(int experts) {
  return 1024 + (size_t)kGwRing + kGwOut + (2 * kGwMaxStages + 4) * 8 + 16 + 2 * 4 * (size_t)(experts + 1);
}

SBN_DEVFN void tc_mma_f16_gw(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(kGwIdesc), "r"(accumulate), "r"(0u)
      : "memory");
}

// tmap_a (the second of two parts p.a_rows rows behind the first), tmap_x: the
// fp16 operands, boxes of 64 columns x 64 rows (128-byte swizzle); tmap_dw: dW as
// [E N, K], boxes of 32 positions x 32 features (64-byte swizzle).
template <int PARTS>
__global__ void __launch_bounds__(kGwThreads, 1)
bwd_dw_grp_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_x,
                  const __grid_constant__ CUtensorMap tmap_dw, const GwParams p) {
  constexpr int kGwABytes = PARTS * kGwPart, kGwStageBytes = kGwABytes + kGwBN * kGwBK * 2;
  constexpr int kGwStages = kGwRing / kGwStageBytes;
  static_assert(kGwStages <= kGwMaxStages, "barriers of the ring");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out = smem + kGwRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(out + kGwOut);
  uint64_t* empty = full + kGwStages;
  uint64_t* acc_full = empty + kGwStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 4);
  int* s_first = s_off + p.grp.experts + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int col_tiles = (p.K + kGwBN - 1) / kGwBN;
  const int per_expert = col_tiles * ((p.N + kGwBM - 1) / kGwBM);
  const int n_tiles = p.grp.experts * per_expert, grid = (int)gridDim.x;

  if (tid == 0) {
    for (int s = 0; s < kGwStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
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
  if (warp == 2) grp_build(p.grp, kGwBK, 1, 0, s_off, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  int used = 0;

  if (warp == 0) {
    const bool lead = elect_one();
    int s = 0;
    uint32_t ph = 1u;
    bool ok = true;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
      const int e = tile / per_expert, local = tile - e * per_expert;
      const int b0 = s_first[e], nst = s_first[e + 1] - b0;
      const int o0 = (local / col_tiles) * kGwBM, k0 = (local % col_tiles) * kGwBN;
      for (int ks = 0; ks < nst; ++ks) {
        if (!mbar_wait_warp(&empty[s], ph)) { ok = false; break; }
        uint8_t* st = smem + (size_t)s * kGwStageBytes;
        const int row = __shfl_sync(0xffffffffu, (b0 + ks) * kGwBK, 0);
        if (lead) {
          // boxes past the last column are zeros
          mbar_arrive_expect_tx(&full[s], (uint32_t)kGwStageBytes);
#pragma unroll
          for (int j = 0; j < PARTS * kGwBM / 64; ++j)
            tma_load_2d(st + j * 8192, &tmap_a, o0 + 64 * (j % (kGwBM / 64)),
                        j < kGwBM / 64 ? row : row + (int)p.a_rows, &full[s]);
#pragma unroll
          for (int j = 0; j < kGwBN / 64; ++j) tma_load_2d(st + kGwABytes + j * 8192, &tmap_x, k0 + 64 * j, row, &full[s]);
        }
        __syncwarp();
        if (++s == kGwStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer: the whole warp runs the loop, one elected lane issues ----
    const bool lead = elect_one();
    const uint32_t base = smem_u32(smem);
    const uint64_t ad0 = sw128_mnmajor_desc(base, 8192u, 1024u), bd0 = sw128_mnmajor_desc(base + kGwABytes, 8192u, 1024u);
    int s = 0;
    uint32_t ph = 0u;
    bool ok = true;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
      const int e = tile / per_expert;
      const int nst = s_first[e + 1] - s_first[e];
      if (nst == 0) continue;
      const int b = used & 1;
      if (!mbar_wait_warp(&acc_empty[b], ((used >> 1) & 1u) ^ 1u)) break;
      const uint32_t d_tmem = tmem + (uint32_t)(b * kGwBN);
      for (int ks = 0; ks < nst; ++ks) {
        if (!mbar_wait_warp(&full[s], ph)) { ok = false; break; }
        tc_fence_after();
        const uint64_t so = (uint64_t)(s * (kGwStageBytes / 16));
        if (lead) {
#pragma unroll
          for (int k = 0; k < PARTS * kGwBK / 16; ++k) {   // 16 rows: two 1 KB atom rows of each operand
            const int part = k % PARTS, rows16 = k / PARTS;
            tc_mma_f16_gw(d_tmem, ad0 + so + (uint64_t)((part * kGwPart + rows16 * 2048) / 16),
                          bd0 + so + (uint64_t)(rows16 * (2048 / 16)), (ks > 0 || k > 0) ? 1u : 0u);
          }
          tc_commit(&empty[s]);
        }
        __syncwarp();
        if (++s == kGwStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (lead) tc_commit(&acc_full[b]);
      __syncwarp();
      ++used;
    }
    for (int j = used - 2; j < used; ++j)
      if (j >= 0) mbar_wait(&acc_full[j & 1], (j >> 1) & 1u);
    __syncwarp();
  } else if (warp >= 4) {
    // ---- epilogue: lane = feature, 32 positions per TMEM load; the second
    // warp of a lane quadrant takes the second half of the positions ----
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    for (int tile = blockIdx.x; tile < n_tiles; tile += grid) {
      const int e = tile / per_expert, local = tile - e * per_expert;
      const bool any = s_first[e + 1] > s_first[e];
      const int b = used & 1;
      const int o = (local / col_tiles) * kGwBM + 32 * q + lane, k0 = (local % col_tiles) * kGwBN;
      const float sc = any && o < p.N ? __ldg(p.scale + (size_t)e * p.N + o) : 0.f;
      if (any) {
        if (!mbar_wait_warp(&acc_full[b], (used >> 1) & 1u)) break;
        ++used;
        tc_fence_after();
      }
      uint16_t* drow = p.dw + ((size_t)e * p.N + o) * p.K;
      const int o_w = o - lane;
      uint8_t* tile_w = out + (warp - 4) * 2048;
#pragma unroll 1
      for (int c = 4 * half; c < 4 * half + 4; ++c) {
        uint32_t r[32];
        if (any) {
          tmem_ld32(tmem + lane_base + (uint32_t)(b * kGwBN + 32 * c), r);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        const int kc = k0 + 32 * c;
        uint32_t o16[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o16[i] = (uint32_t)f32_to_bf16_bits(__fmul_rn(sc, __uint_as_float(r[2 * i]))) |
                   ((uint32_t)f32_to_bf16_bits(__fmul_rn(sc, __uint_as_float(r[2 * i + 1]))) << 16);
        if (o_w + 32 <= p.N && kc < p.K) {
          // through shared memory, so that whole rows of a box leave at once
          if (lane == 0) tma_store_wait_read0();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(tile_w + epi_piece(lane, i)) =
                make_uint4(o16[4 * i], o16[4 * i + 1], o16[4 * i + 2], o16[4 * i + 3]);
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) tma_store_2d(&tmap_dw, kc, e * p.N + o_w, tile_w);
        } else if (o < p.N && kc < p.K) {   // the last features, whose box would reach into the next expert
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
    if (lane == 0) tma_store_wait_all();
    griddep_launch_dependents();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kBxTmemCols) : "memory");
  }
}

}  // namespace sbn
