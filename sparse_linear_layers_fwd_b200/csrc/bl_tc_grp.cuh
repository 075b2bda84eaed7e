// Contraction of rows grouped by expert on the 5th-generation tensor cores,
// with the layer's epilogue, straight from the packed weights.
//
// "Microsoft BitNet 1.58: The Era of 1-Bit Large Language Models", section
// "The BitLinear Layer", fourth and fifth operations, for a set of layers
// (experts) of one shape: row r of expert e gets f(acc gamma_e s_r / 127 +
// bias_e) + residual. Without offsets it is one layer over all rows.
//
// A persistent CTA per SM walks the tiles of the work list (grp.cuh): 128
// output features x up to 192 rows of one expert, an expert's rows split into
// equal tiles (of 32-row chunks; the MMA's N is a multiple of 16). The packed
// weights are read once per tile and expanded on the way to the MMA, since an
// expert sees few rows: expanding them in memory first would cost as much as
// the product itself at 500 rows.
//
// The expanded weights go from the producers' registers straight into tensor
// memory, as the MMA's A operand (lane = feature, 32-bit column = four
// positions): they never touch shared memory, whose bandwidth the activations
// need (read by the MMA at 64 bytes a cycle, written by TMA at the same rate).
//   warp 0      TMA of the activation rows (boxes of 64 and 16 rows), blocks of
//               128 positions;
//   warp 1      TMEM allocation and the MMA warp;
//   warp 2      the work list, then TMA of the packed rows (codes and keep
//               bits of 128 features x 256 positions) into a ring of their own;
//   warps 4-15  producers: three groups of four warps, one for each A slot,
//               take the 128-position blocks in turn; a thread expands its
//               feature's positions (bl_gemv.cuh's expansion) into 32 registers
//               and stores them with tcgen05.st. A slot belongs to one group, so
//               that a wait by parity can never be two rounds behind or ahead;
//   warps 16-23 epilogue (epi_tile.cuh), two per TMEM lane quadrant, the
//               first taking the first half of a tile's 32-row chunks.
// The loops of the MMA and TMA warps are run by whole warps and only the
// instructions themselves by one elected lane: addresses and descriptors then
// live in uniform registers, and eight MMAs are issued in 190 cycles instead
// of 840. Every lane waits on a barrier itself, which is faster than one lane
// and a shuffle.
// TMEM: two accumulators of 192 columns, so that the epilogue hides behind the
// next tile, and three A slots of 32 columns (a 128-position block each).
// Measured at 16384 rows (30 of 32 experts, K = 2048, N_out = 2816, 6:8, with the
// quantization) and at 256 rows of 64 experts (K = 2048, N_out = 1408, 2:4),
// whole calls, the inputs changed from call to call:
//   this split                                         151 to 155 us, 39.1 us
//   the even codes masked group by group, not once
//   a span                                             154 to 156 us, 40.2 us
// On an earlier build that took 138 and 43.2 us on one set of inputs:
//   160-column accumulators, one ring of three 256-position
//   stages for both operands                                  153 us, 39 us
//   one accumulator of 256 columns, its epilogue exposed      150 us, 43.6 us
//   four groups of producers and slots (72 registers)         142 us, 42 us
// What bounds it: a block costs 760 to 1040 cycles, of which the MMAs need 384
// at 192 rows. Half of the issue slots are taken (the expansion's permutes and
// the epilogue share the integer pipe, 56 % busy), so that the MMA warp's own
// instructions wait for theirs: a barrier that is already complete costs it
// 130 cycles, four MMAs and their commits 210 to 260. A first look at the next
// block's barriers ahead of the MMAs, deeper rings and wider boxes of packed
// rows changed nothing.
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
constexpr int kTgBN = 192;
constexpr int kTgBlocks = 5;                   // activation ring, blocks of 128 positions
constexpr int kTgBlockBytes = kTgBN * 128;
constexpr int kTgSlots = 3;                    // A slots in TMEM, a block and a producer group each
constexpr uint32_t kTgACol = 2 * kTgBN;        // after the accumulators
static_assert(kTgACol + 32 * kTgSlots <= kTcTmemCols, "accumulators and A slots fit in TMEM");
static_assert(kTgBlockBytes % 1024 == 0, "swizzled tiles stay 1024-byte aligned");
constexpr int kTgSpan = 2;                     // blocks of a stage of packed rows
constexpr int kTgPackedBytes = kTgBM * (24 + 16) * kTgSpan;   // a stage, at most (6:8; n == m: 32 and no keep bits)
constexpr int kTgPacked = 5;                   // their ring: a slot is free only when its stage is expanded
constexpr int kTgThreads = 768;
constexpr int kTgEpiWarp = 16;                 // first epilogue warp
constexpr int kTgSelCopies = 8;
constexpr int kTgEpiWarps = 8;
constexpr int kTgYBuf = kTgEpiWarps * (4096 + 128);
constexpr int kTgBars = 2 * (kTgBlocks + kTgSlots + 2) + 3 * kTgPacked;
constexpr int kTgList = 64;                    // tiles of a CTA whose place is worked out ahead
constexpr uint32_t kTgIdesc0 = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTgBM >> 4) << 24);

__host__ __device__ inline size_t tg_smem_bytes(int experts) {
  return 1024 + (size_t)kTgBlocks * kTgBlockBytes + (size_t)kTgPacked * kTgPackedBytes + kTgYBuf + 256 * 4 * kTgSelCopies +
         16 * kTgList + kTgBars * 8 + 4 + 2 * 4 * (size_t)(experts + 1);
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
  const int size = ((n + parts - 1) / parts + 31) / 32 * 32;   // whole chunks of the epilogue
  const int tt = local / row_tiles;
  t.row0 = (local - tt * row_tiles) * bm;
  t.tok0 = lo + tt * size;
  t.tok_end = min(hi, t.tok0 + size);
  const int have = t.tok_end - t.tok0;
  t.nmma = have > 0 ? (have + step - 1) / step * step : 0;
  return t;
}

// A from tensor memory, B from shared memory.
SBN_DEVFN void tc_mma_i8_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(0u)
      : "memory");
}
// 16 columns of this warp's 32 lanes from registers, and the wait for all such.
SBN_DEVFN void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
SBN_DEVFN void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// The k-th tile of this CTA: from the list (`len` entries), worked out on the
// spot behind it. BM, BN, STEP: tg_tile's.
template <int BM, int BN, int STEP>
SBN_DEVFN TgTile tg_get(const int4* list, int len, const int* off, const int* first, const GrpParams& g, int k,
                        int row_tiles) {
  if (k >= len) return tg_tile(off, first, g, (int)blockIdx.x + k * (int)gridDim.x, row_tiles, BM, BN, STEP);
  const int4 v = list[k];
  const int have = v.w - v.z;
  return TgTile{v.x, v.y, v.z, v.w, have > 0 ? (have + STEP - 1) / STEP * STEP : 0};
}
// The list, by all threads of the CTA: its first `len` tiles of `count`.
template <int BM, int BN, int STEP>
SBN_DEVFN void tg_list(int4* list, int len, const int* off, const int* first, const GrpParams& g, int count,
                       int row_tiles) {
  for (int k = (int)threadIdx.x; k < min(count, len); k += (int)blockDim.x) {
    const TgTile t = tg_tile(off, first, g, (int)blockIdx.x + k * (int)gridDim.x, row_tiles, BM, BN, STEP);
    list[k] = make_int4(t.e, t.row0, t.tok0, t.tok_end);
  }
}

// Eight positions (group I of a span) as in bl_gemv.cuh's gv_expand, for m = 4
// and 8. ew: the code words masked with 0x33333333, once for the span instead
// of once for each group: a selector's nibbles past the group's then pick
// some byte of the table, and no position takes its value (a pruned position
// takes the odd codes' last byte, whose selectors are masked group by group).
template <int CB, int I>
SBN_DEVFN void tg_expand8(const uint32_t (&cw)[CB], const uint32_t (&ew)[CB], const uint32_t (&mw)[2],
                          const uint32_t* sel, uint32_t& w0, uint32_t& w1) {
  constexpr int kOff = 4 * CB * I, i = kOff / 32, s = kOff % 32;
  constexpr uint32_t kMask = CB == 1 ? 0x3u : CB == 2 ? 0x33u : 0x333u;
  const uint32_t m8 = gv_prmt(mw[I / 4], 0u, 0x4440u | (I % 4));
  uint32_t e;
  if constexpr (s + 4 * CB <= 32) e = ew[i] >> s;
  else e = __funnelshift_r(ew[i], ew[i + 1], s);
  const uint32_t ev = gv_prmt(kCodeByteTable, 0u, e);
  const uint32_t od = gv_prmt(kCodeByteTable, 0u, gv_field<kOff + 2, kMask, CB>(cw));
  gv_place(sel[m8 * kTgSelCopies], ev, od, w0, w1);
}

// 64 positions (one span of bl_gemv.cuh) -> 16 words of int8.
template <int MM, int CB, bool DENSE>
SBN_DEVFN void tg_expand64(const uint32_t (&cw)[CB], const uint32_t (&mw)[2], const uint32_t* sel, uint32_t* w) {
  if constexpr (!DENSE && MM != 16) {
    uint32_t ew[CB];
#pragma unroll
    for (int i = 0; i < CB; ++i) ew[i] = cw[i] & 0x33333333u;
    tg_expand8<CB, 0>(cw, ew, mw, sel, w[0], w[1]);
    tg_expand8<CB, 1>(cw, ew, mw, sel, w[2], w[3]);
    tg_expand8<CB, 2>(cw, ew, mw, sel, w[4], w[5]);
    tg_expand8<CB, 3>(cw, ew, mw, sel, w[6], w[7]);
    tg_expand8<CB, 4>(cw, ew, mw, sel, w[8], w[9]);
    tg_expand8<CB, 5>(cw, ew, mw, sel, w[10], w[11]);
    tg_expand8<CB, 6>(cw, ew, mw, sel, w[12], w[13]);
    tg_expand8<CB, 7>(cw, ew, mw, sel, w[14], w[15]);
  } else {
    gv_expand<MM, CB, DENSE, 0, kTgSelCopies>(cw, mw, sel, w[0], w[1]);
    gv_expand<MM, CB, DENSE, 1, kTgSelCopies>(cw, mw, sel, w[2], w[3]);
    gv_expand<MM, CB, DENSE, 2, kTgSelCopies>(cw, mw, sel, w[4], w[5]);
    gv_expand<MM, CB, DENSE, 3, kTgSelCopies>(cw, mw, sel, w[6], w[7]);
    gv_expand<MM, CB, DENSE, 4, kTgSelCopies>(cw, mw, sel, w[8], w[9]);
    gv_expand<MM, CB, DENSE, 5, kTgSelCopies>(cw, mw, sel, w[10], w[11]);
    gv_expand<MM, CB, DENSE, 6, kTgSelCopies>(cw, mw, sel, w[12], w[13]);
    gv_expand<MM, CB, DENSE, 7, kTgSelCopies>(cw, mw, sel, w[14], w[15]);
  }
}

template <int MM, int CB, bool DENSE>
__global__ void __launch_bounds__(kTgThreads, 1)
bl_tc_grp_kernel(const __grid_constant__ CUtensorMap tmap_x64, const __grid_constant__ CUtensorMap tmap_x16,
                 const __grid_constant__ CUtensorMap tmap_c, const __grid_constant__ CUtensorMap tmap_m,
                 const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_z,
                 const TgParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* packed = smem + (size_t)kTgBlocks * kTgBlockBytes;
  uint8_t* ybuf = packed + kTgPacked * kTgPackedBytes;
  uint32_t* s_sel = reinterpret_cast<uint32_t*>(ybuf + kTgYBuf);   // [256][kTgSelCopies]
  int4* s_list = reinterpret_cast<int4*>(s_sel + 256 * kTgSelCopies);
  uint64_t* b_full = reinterpret_cast<uint64_t*>(s_list + kTgList);
  uint64_t* b_empty = b_full + kTgBlocks;
  uint64_t* a_full = b_empty + kTgBlocks;
  uint64_t* a_empty = a_full + kTgSlots;
  uint64_t* p_full = a_empty + kTgSlots;
  uint64_t* p_empty = p_full + 2 * kTgPacked;
  uint64_t* acc_full = p_empty + kTgPacked;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 1);
  int* s_first = s_off + p.grp.experts + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nkb = p.K / 128;            // 128-position blocks
  const int nst = (nkb + kTgSpan - 1) / kTgSpan;   // stages of packed rows
  const int row_tiles = (p.N + kTgBM - 1) / kTgBM;

  if (tid == 0) {
    for (int s = 0; s < kTgBlocks; ++s) {
      mbar_init(&b_full[s], 1);
      mbar_init(&b_empty[s], 1);
    }
    for (int s = 0; s < kTgSlots; ++s) {
      mbar_init(&a_full[s], 4);   // a group's warps
      mbar_init(&a_empty[s], 1);
    }
    for (int s = 0; s < kTgPacked; ++s) {
      mbar_init(&p_full[s], 1);
      mbar_init(&p_full[s + kTgPacked], 1);
      mbar_init(&p_empty[s], 4 * kTgSpan);   // the warps of a stage's blocks
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kTgEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmap_x64);
    tma_prefetch_map(&tmap_x16);
    tma_prefetch_map(&tmap_c);
    if (!DENSE) tma_prefetch_map(&tmap_m);
    if (p.aligned) tma_prefetch_map(&tmap_y);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(s_tmem)),
                 "r"(kTcTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (!DENSE) {
    for (int i = tid; i < 256 * kTgSelCopies; i += blockDim.x) s_sel[i] = gv_selector((uint32_t)(i / kTgSelCopies));
  }
  griddep_wait();
  if (warp == 2) grp_build(p.grp, kTgBN, row_tiles, 0, s_off, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int n_tiles = s_first[p.grp.experts];
  const int count = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  tg_list<kTgBM, kTgBN, 16>(s_list, kTgList, s_off, s_first, p.grp, count, row_tiles);
  __syncthreads();
  int used = 0;   // tiles this role has worked on

  if (warp == 0) {
    // ---- TMA of the activation rows ----
    const bool lead = elect_one();
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int k = 0; k < count && ok; ++k) {
      const TgTile t = tg_get<kTgBM, kTgBN, 16>(s_list, kTgList, s_off, s_first, p.grp, k, row_tiles);
      if (!t.nmma) continue;
      const int nmma = __shfl_sync(0xffffffffu, t.nmma, 0), tok0 = __shfl_sync(0xffffffffu, t.tok0, 0);
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait_warp(&b_empty[s], ph)) { ok = false; break; }
        uint8_t* dst = smem + (size_t)s * kTgBlockBytes;
        if (lead) {
          mbar_arrive_expect_tx(&b_full[s], (uint32_t)nmma * 128u);
          int r = 0;
          for (; r + 64 <= nmma; r += 64) tma_load_2d(dst + r * 128, &tmap_x64, kb * 128, tok0 + r, &b_full[s]);
          for (; r < nmma; r += 16) tma_load_2d(dst + r * 128, &tmap_x16, kb * 128, tok0 + r, &b_full[s]);
        }
        __syncwarp();
        if (++s == kTgBlocks) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 2) {
    // ---- TMA of the packed rows ----
    const bool lead = elect_one();
    int s = 0, f = 0;   // slot, and barrier of its arrival
    uint32_t ph = 1;
    bool ok = true;
    for (int k = 0; k < count && ok; ++k) {
      const TgTile t = tg_get<kTgBM, kTgBN, 16>(s_list, kTgList, s_off, s_first, p.grp, k, row_tiles);
      if (!t.nmma) continue;
      // rows past the expert's are expanded, never stored
      const int row = __shfl_sync(0xffffffffu, t.e * p.N + t.row0, 0);
      for (int ks = 0; ks < nst; ++ks) {
        if (!mbar_wait_warp(&p_empty[s], ph)) { ok = false; break; }
        uint8_t* dst = packed + s * kTgPackedBytes;
        if (lead) {
          mbar_arrive_expect_tx(&p_full[f], (uint32_t)(kTgBM * kTgSpan * (8 * CB + (DENSE ? 0 : 16))));
          tma_load_2d(dst, &tmap_c, ks * 16 * CB, row, &p_full[f]);
          if (!DENSE) tma_load_2d(dst + kTgBM * kTgSpan * 8 * CB, &tmap_m, ks * kTgSpan * 16, row, &p_full[f]);
        }
        __syncwarp();
        if (++f == 2 * kTgPacked) f = 0;
        if (++s == kTgPacked) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer: the whole warp runs the loop (addresses and descriptors
    // stay in uniform registers), one elected lane issues ----
    const bool lead = elect_one();
    const uint64_t bdesc0 = sw128_kmajor_desc(smem_u32(smem));
    int s = 0, a = 0;
    uint32_t ph = 0, pa = 0;
    bool ok = true;
    TgTile t = count ? tg_get<kTgBM, kTgBN, 16>(s_list, kTgList, s_off, s_first, p.grp, 0, row_tiles) : TgTile{};
    for (int k = 0; k < count && ok; ++k) {
      const int nmma = t.nmma;
      if (k + 1 < count) t = tg_get<kTgBM, kTgBN, 16>(s_list, kTgList, s_off, s_first, p.grp, k + 1, row_tiles);
      if (!nmma) continue;
      const uint32_t idesc = __shfl_sync(0xffffffffu, kTgIdesc0 | ((uint32_t)(nmma >> 3) << 17), 0);
      const int b = used & 1;
      if (!mbar_wait_warp(&acc_empty[b], ((used >> 1) & 1u) ^ 1u)) break;
      const uint32_t d_tmem = tmem + (uint32_t)(b * kTgBN);
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait_warp(&b_full[s], ph, &a_full[a], pa)) { ok = false; break; }
        tc_fence_after();
        const uint64_t bdesc = bdesc0 + (uint64_t)(s * (kTgBlockBytes / 16));
        const uint32_t a_tmem = tmem + kTgACol + 32u * (uint32_t)a;
        if (lead) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tc_mma_i8_ta(d_tmem, a_tmem + 8u * (uint32_t)i, bdesc + (uint64_t)(2 * i), idesc,
                         (kb > 0 || i > 0) ? 1u : 0u);
          tc_commit(&a_empty[a]);
          tc_commit(&b_empty[s]);
        }
        __syncwarp();
        if (++s == kTgBlocks) {
          s = 0;
          ph ^= 1u;
        }
        if (++a == kTgSlots) {
          a = 0;
          pa ^= 1u;
        }
      }
      if (lead) tc_commit(&acc_full[b]);
      __syncwarp();
      ++used;
    }
    // the last commits before TMEM is freed (also on the abort path)
    for (int j = used - 2; j < used; ++j)
      if (j >= 0) mbar_wait(&acc_full[j & 1], (j >> 1) & 1u);
    __syncwarp();
  } else if (warp >= 4 && warp < kTgEpiWarp) {
    // ---- producers: thread = feature 32 q + lane, group g takes the blocks with
    // index = g (mod 3) over all tiles, into slot g ----
    const int q = warp & 3, g = (warp - 4) >> 2;
    const int i = 32 * q + lane;
    const uint32_t* sel = s_sel + (lane & (kTgSelCopies - 1));
    const uint32_t a_tmem = tmem + kTgACol + 32u * (uint32_t)g + ((uint32_t)(32 * q) << 16);
    int it = 0, blk = 0;   // stages and blocks before the tile
    uint32_t ph = 1u;
    bool ok = true;
    for (int k = 0; k < count && ok; ++k) {
      const TgTile t = tg_get<kTgBM, kTgBN, 16>(s_list, kTgList, s_off, s_first, p.grp, k, row_tiles);
      if (!t.nmma) continue;
      for (int kb = (g - blk % kTgSlots + kTgSlots) % kTgSlots; kb < nkb; kb += kTgSlots, ph ^= 1u) {
        // Two arrival barriers for a packed slot, taken in turn: a group may look
        // before the slot's previous stage has landed, but never before the one
        // before that (it has seen the MMA of the block 2 kTgSlots back).
        const int st = it + kb / kTgSpan, ps = st % kTgPacked, j = kb % kTgSpan;
        if (!mbar_wait_warp(&p_full[st % (2 * kTgPacked)], (uint32_t)(st / (2 * kTgPacked)) & 1u)) { ok = false; break; }
        const uint2* cp = reinterpret_cast<const uint2*>(packed + ps * kTgPackedBytes + (i * kTgSpan + j) * 8 * CB);
        uint32_t cw[2][CB];
#pragma unroll
        for (int h = 0; h < CB; ++h) {
          const uint2 c2 = cp[h];
          cw[2 * h / CB][2 * h % CB] = c2.x;
          cw[(2 * h + 1) / CB][(2 * h + 1) % CB] = c2.y;
        }
        uint4 mv = make_uint4(0u, 0u, 0u, 0u);
        if (!DENSE)
          mv = *reinterpret_cast<const uint4*>(packed + ps * kTgPackedBytes + kTgBM * kTgSpan * 8 * CB + (i * kTgSpan + j) * 16);
        const uint32_t m0[2] = {mv.x, mv.y}, m1[2] = {mv.z, mv.w};
        uint32_t w[16], v[16];
        tg_expand64<MM, CB, DENSE>(cw[0], m0, sel, w);
        tg_expand64<MM, CB, DENSE>(cw[1], m1, sel, v);
        if (!mbar_wait_warp(&a_empty[g], ph)) { ok = false; break; }
        tc_fence_after();
        tmem_st16(a_tmem, w);
        tmem_st16(a_tmem + 16u, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&a_full[g]);
          // the packed rows only now, when what was loaded of them has been used:
          // handed back right behind the loads, they were overwritten before every
          // lane's loads had been done. The last block counts for those behind it.
          for (int n = kb + 1 == nkb ? j : kTgSpan - 1; n < kTgSpan; ++n) mbar_arrive(&p_empty[ps]);
        }
      }
      it += nst;
      blk += nkb;
    }
  } else if (warp >= kTgEpiWarp) {
    // ---- epilogue ----
    const int q = warp & 3;
    const bool second = warp >= kTgEpiWarp + 4;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    EpiTile et{reinterpret_cast<uint16_t*>(ybuf + (size_t)(warp - kTgEpiWarp) * 4096),
               reinterpret_cast<float*>(ybuf + kTgEpiWarps * 4096) + 32 * (warp - kTgEpiWarp), 0};
    const EpiOut out{&tmap_y, &tmap_z, p.y, p.N, p.grp.rows, p.aligned != 0};
    for (int k = 0; k < count; ++k) {
      const TgTile t = tg_get<kTgBM, kTgBN, 16>(s_list, kTgList, s_off, s_first, p.grp, k, row_tiles);
      if (!t.nmma) continue;
      const int b = used & 1;
      const int row_w = t.row0 + 32 * q;
      const float gm = __ldg(p.gamma + t.e);
      const float bias = (p.ep.bias && row_w + lane < p.N) ? __ldg(p.ep.bias + (size_t)t.e * p.N + row_w + lane) : 0.f;
      const int chunks = (t.tok_end - t.tok0 + 31) / 32;
      const int c_first = second ? (chunks + 1) / 2 : 0, c_end = second ? chunks : (chunks + 1) / 2;
      const int tok_w = t.tok0 + 32 * c_first;
      uint4 res[4];
      epi_load_residual(p.ep, out, row_w, tok_w, t.tok_end, lane, res);
      float xs_n = tok_w + lane < t.tok_end ? __ldg(p.xs + tok_w + lane) : 0.f;
      if (!mbar_wait_warp(&acc_full[b], (used >> 1) & 1u)) break;
      ++used;
      tc_fence_after();
#pragma unroll 1
      for (int c = c_first; c < c_end; ++c) {
        const int tok = t.tok0 + 32 * c;
        const float sc = __fdiv_rn(__fmul_rn(gm, xs_n), 127.0f);
        xs_n = tok + 32 + lane < t.tok_end ? __ldg(p.xs + tok + 32 + lane) : 0.f;
        epi_chunk(p.ep, out, et, tmem + lane_base + (uint32_t)(b * kTgBN + 32 * c), sc, bias, row_w, tok, t.tok_end,
                  c + 1 < c_end ? tok + 32 : -1, lane, res, c + 1 < c_end ? nullptr : &acc_empty[b]);
      }
      if (c_first == c_end && lane == 0) mbar_arrive(&acc_empty[b]);   // no chunk for this warp
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
