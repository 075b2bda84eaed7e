// Contraction of rows grouped by expert on the 5th-generation tensor cores,
// with the layer's epilogue, straight from the packed weights.
//
// "Microsoft BitNet 1.58: The Era of 1-Bit Large Language Models", section
// "The BitLinear Layer", fourth and fifth operations, for a set of layers
// (experts) of one shape: row r of expert e gets f(acc gamma_e s_r / 127 +
// bias_e) + residual. Without offsets it is one layer over all rows.
//
// A persistent CTA per SM walks the tiles of the work list (grp.cuh): 128
// output features x up to 256 rows of one expert, an expert's rows split into
// equal tiles (a multiple of 16 rows each, the MMA's N). The weights are
// expanded in shared memory by eight producer warps, since an expert sees few
// rows: writing the expanded weights to memory and reading them back would
// cost as much as the product itself at 500 rows.
//   warp 0      TMA of the activation rows (boxes of 64 and 16 rows);
//   warp 1      TMEM allocation and the MMA thread;
//   warp 2      the work list;
//   warps 4-11  producers (bl_tc.cuh), with the expansion of bl_gemv.cuh;
//   warps 12-15 epilogue (epi_tile.cuh).
// Rows of the next expert that share a box are loaded and multiplied, never
// stored. All waits are bounded in time.
#pragma once

#include <cuda.h>

#include "async.cuh"
#include "bl_gemv.cuh"
#include "bl_tc.cuh"
#include "common.cuh"
#include "epi_tile.cuh"
#include "grp.cuh"

namespace sbn {

constexpr int kTgBM = 128;
constexpr int kTgBN = 256;
constexpr int kTgStages = 4;
constexpr int kTgABytes = kTgBM * 128;
constexpr int kTgStageBytes = kTgABytes + kTgBN * 128;
constexpr int kTgSelCopies = 4;
constexpr int kTgYBuf = (kTcEpilogue / 32) * 4096;
constexpr uint32_t kTgIdesc0 = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTgBM >> 4) << 24);

__host__ __device__ inline size_t tg_smem_bytes(int experts) {
  return 1024 + (size_t)kTgStages * kTgStageBytes + kTgYBuf + 256 * 8 * kTgSelCopies + (2 * kTgStages + 4) * 8 + 16 +
         2 * 4 * (size_t)(experts + 1);
}

struct TgParams {
  const uint8_t* codes;   // [E, N_out, cstride]
  const uint8_t* meta;
  const float* xs;        // [R]
  const float* gamma;     // [E]
  uint16_t* y;
  EpiParams ep;
  GrpParams grp;
  int K, N;
  int cstride, mstride;
  int aligned;            // tile stores (16-byte rows of y, z and the residual)
};

// A tile of the work list.
struct TgTile {
  int e, row0, tok0, tok_end, nmma;   // nmma = 0: nothing to do
};

SBN_DEVFN TgTile tg_tile(const int* off, const int* first, const GrpParams& g, int tile, int row_tiles, int bm, int bn,
                         int step) {
  TgTile t;
  t.e = grp_find(first, g.experts, tile);
  const int local = tile - first[t.e];
  const int lo = off[t.e], hi = off[t.e + 1], n = hi - lo;
  const int parts = (n + bn - 1) / bn;
  const int size = ((n + parts - 1) / parts + step - 1) / step * step;
  const int tt = local / row_tiles;
  t.row0 = (local - tt * row_tiles) * bm;
  t.tok0 = lo + tt * size;
  t.tok_end = min(hi, t.tok0 + size);
  const int have = t.tok_end - t.tok0;
  t.nmma = have > 0 ? (have + step - 1) / step * step : 0;
  return t;
}

SBN_DEVFN void tc_mma_i8_n(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(0u)
      : "memory");
}

// 64 positions (one span of bl_gemv.cuh) -> 16 words of int8.
template <int MM, int CB, bool DENSE>
SBN_DEVFN void tg_expand64(const uint32_t (&cw)[CB], const uint32_t (&mw)[2], const uint2* sel, uint32_t (&w)[16]) {
  gv_expand<MM, CB, DENSE, 0, kTgSelCopies>(cw, mw, sel, w[0], w[1]);
  gv_expand<MM, CB, DENSE, 1, kTgSelCopies>(cw, mw, sel, w[2], w[3]);
  gv_expand<MM, CB, DENSE, 2, kTgSelCopies>(cw, mw, sel, w[4], w[5]);
  gv_expand<MM, CB, DENSE, 3, kTgSelCopies>(cw, mw, sel, w[6], w[7]);
  gv_expand<MM, CB, DENSE, 4, kTgSelCopies>(cw, mw, sel, w[8], w[9]);
  gv_expand<MM, CB, DENSE, 5, kTgSelCopies>(cw, mw, sel, w[10], w[11]);
  gv_expand<MM, CB, DENSE, 6, kTgSelCopies>(cw, mw, sel, w[12], w[13]);
  gv_expand<MM, CB, DENSE, 7, kTgSelCopies>(cw, mw, sel, w[14], w[15]);
}

template <int MM, int CB, bool DENSE>
__global__ void __launch_bounds__(kTcThreads, 1)
bl_tc_grp_kernel(const __grid_constant__ CUtensorMap tmap_x64, const __grid_constant__ CUtensorMap tmap_x16,
                 const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_z,
                 const TgParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ybuf = smem + (size_t)kTgStages * kTgStageBytes;
  uint2* s_sel = reinterpret_cast<uint2*>(ybuf + kTgYBuf);   // [256][kTgSelCopies]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_sel + 256 * kTgSelCopies);
  uint64_t* empty = full + kTgStages;
  uint64_t* acc_full = empty + kTgStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 4);
  int* s_first = s_off + p.grp.experts + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nkb = p.K / 128;
  const int row_tiles = (p.N + kTgBM - 1) / kTgBM;

  if (tid == 0) {
    for (int s = 0; s < kTgStages; ++s) {
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
                 "r"(kTcTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (!DENSE) {
    for (int i = tid; i < 256 * kTgSelCopies; i += blockDim.x) s_sel[i] = gv_selector_pair((uint32_t)(i / kTgSelCopies));
  }
  griddep_wait();
  if (warp == 2) grp_build(p.grp, kTgBN, row_tiles, 0, s_off, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int n_tiles = s_first[p.grp.experts];
  const int grid = (int)gridDim.x;
  int used = 0;   // tiles this role has worked on

  if (warp == 0) {
    // ---- TMA of the activation rows ----
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
        const TgTile t = tg_tile(s_off, s_first, p.grp, tile, row_tiles, kTgBM, kTgBN, 16);
        if (!t.nmma) continue;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % kTgStages;
          if (!mbar_wait(&empty[s], ((it / kTgStages) & 1u) ^ 1u)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[s], (uint32_t)t.nmma * 128u);
          uint8_t* dst = smem + (size_t)s * kTgStageBytes + kTgABytes;
          int r = 0;
          for (; r + 64 <= t.nmma; r += 64) tma_load_2d(dst + r * 128, &tmap_x64, kb * 128, t.tok0 + r, &full[s]);
          for (; r < t.nmma; r += 16) tma_load_2d(dst + r * 128, &tmap_x16, kb * 128, t.tok0 + r, &full[s]);
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
        const TgTile t = tg_tile(s_off, s_first, p.grp, tile, row_tiles, kTgBM, kTgBN, 16);
        if (!t.nmma) continue;
        const uint32_t idesc = kTgIdesc0 | ((uint32_t)(t.nmma >> 3) << 17);
        const int b = used & 1;
        if (!mbar_wait(&acc_empty[b], ((used >> 1) & 1u) ^ 1u)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(b * kTgBN);
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % kTgStages;
          if (!mbar_wait(&full[s], (it / kTgStages) & 1u)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + (size_t)s * kTgStageBytes);
          const uint64_t adesc = sw128_kmajor_desc(a_addr), bdesc = sw128_kmajor_desc(a_addr + kTgABytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_i8_n(d_tmem, adesc + (uint64_t)(2 * k), bdesc + (uint64_t)(2 * k), idesc, (kb > 0 || k > 0) ? 1u : 0u);
          tc_commit(&empty[s]);
        }
        tc_commit(&acc_full[b]);
        ++used;
      }
      // the last commits before TMEM is freed (also on the abort path)
      for (int j = used - 2; j < used; ++j)
        if (j >= 0) mbar_wait(&acc_full[j & 1], (j >> 1) & 1u);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ---- producers: thread (i, h) expands positions 64 h .. of row i ----
    const int pi = tid - 128, i = pi & 127, h = pi >> 7;
    const uint2* sel = s_sel + (lane & (kTgSelCopies - 1));
    int it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += grid) {
      const TgTile t = tg_tile(s_off, s_first, p.grp, tile, row_tiles, kTgBM, kTgBN, 16);
      if (!t.nmma) continue;
      const int row = min(t.row0 + i, p.N - 1);   // rows past N repeat the last one; not stored
      const size_t wrow = (size_t)t.e * p.N + row;
      const uint8_t* crow = p.codes + wrow * p.cstride + h * 4 * CB;
      const uint8_t* mrow = DENSE ? nullptr : p.meta + wrow * p.mstride + h * 8;
      uint32_t cn[CB], mn[2] = {0u, 0u};
      auto load = [&](int kb) {
        if (kb < nkb) {
          const uint32_t* cp = reinterpret_cast<const uint32_t*>(crow + (size_t)kb * 8 * CB);
#pragma unroll
          for (int q = 0; q < CB; ++q) cn[q] = __ldg(cp + q);
          if (!DENSE) {
            const uint2 m = __ldg(reinterpret_cast<const uint2*>(mrow + (size_t)kb * 16));
            mn[0] = m.x;
            mn[1] = m.y;
          }
        }
      };
      load(0);
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int s = it % kTgStages;
        uint32_t cw[CB], mw[2] = {mn[0], mn[1]};
#pragma unroll
        for (int q = 0; q < CB; ++q) cw[q] = cn[q];
        load(kb + 1);
        uint32_t w[16];
        tg_expand64<MM, CB, DENSE>(cw, mw, sel, w);
        int got = 1;
        if (lane == 0) got = mbar_wait(&empty[s], ((it / kTgStages) & 1u) ^ 1u) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) { ok = false; break; }
        uint8_t* arow = smem + (size_t)s * kTgStageBytes + (size_t)i * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(arow + (((4 * h + u) ^ (i & 7)) << 4)) =
              make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
  } else if (warp >= 12) {
    // ---- epilogue ----
    const int q = warp & 3;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    EpiTile et{reinterpret_cast<uint16_t*>(ybuf + (size_t)(warp - 12) * 4096), 0};
    const EpiOut out{&tmap_y, &tmap_z, p.y, p.N, p.grp.rows, p.aligned != 0};
    for (int tile = blockIdx.x; tile < n_tiles; tile += grid) {
      const TgTile t = tg_tile(s_off, s_first, p.grp, tile, row_tiles, kTgBM, kTgBN, 16);
      if (!t.nmma) continue;
      const int b = used & 1;
      const int row_w = t.row0 + 32 * q;
      const float gm = __ldg(p.gamma + t.e);
      const float bias = (p.ep.bias && row_w + lane < p.N) ? __ldg(p.ep.bias + (size_t)t.e * p.N + row_w + lane) : 0.f;
      const int chunks = (t.tok_end - t.tok0 + 31) / 32;
      uint4 res[4];
      epi_load_residual(p.ep, out, row_w, t.tok0, t.tok_end, lane, res);
      int got = 1;
      if (lane == 0) got = mbar_wait(&acc_full[b], (used >> 1) & 1u) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      ++used;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int tok = t.tok0 + 32 * c;
        const float sc = tok + lane < t.tok_end ? __fdiv_rn(__fmul_rn(gm, __ldg(p.xs + tok + lane)), 127.0f) : 0.f;
        uint32_t r[32];
        tmem_ld32(tmem + lane_base + (uint32_t)(b * kTgBN + 32 * c), r);
        epi_chunk(p.ep, out, et, r, sc, bias, row_w, tok, t.tok_end, c + 1 < chunks ? tok + 32 : -1, lane, res);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
    if (lane == 0) tma_store_wait_all();
    griddep_launch_dependents();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTcTmemCols) : "memory");
  }
}

}  // namespace sbn
