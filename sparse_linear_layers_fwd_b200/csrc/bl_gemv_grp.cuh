// Decode contraction (R <= 16 rows in all) with the layer's epilogue, over the
// packed weights of one layer or of the experts that have rows.
//
// "Microsoft BitNet 1.58: The Era of 1-Bit Large Language Models", section
// "bitnet.cpp: Matrix-Free Inference", as in bl_gemv.cuh, whose expansion and
// fragment layout this kernel shares: y = f(acc gamma_e s_r / 127 + bias) +
// residual, for the rows r of every expert e. Bound by the packed bytes of
// the experts that have rows (at most 16 of them, however many there are).
//
// One CTA of 1024 threads per SM owns a contiguous range of the work list,
// all 16-row tiles of all experts with rows. The producer warp reads the
// offsets, writes the list of experts with rows (sanitized as in grp.cuh) to
// shared memory, and streams tiles into a ring of slots with one bulk copy of
// codes and one of keep bits each; a range longer than the ring (an expert
// set whose bytes exceed the SM's shared memory) reuses slots. The 31 consumer
// warps take (tile, 256 positions) items in turn and add their partial sums
// into the slot's accumulators; the warp that completes a tile's last item
// runs its epilogue and hands the slot back, so a tile's output is written
// while later tiles are still arriving and no barrier ends the kernel.
// Measured, captured calls: 6.1 us for one token (layer of 6912 x 2560, 6:8, 5.5
// MB), of which launch, prologue and selector tables are about 4; 9.7 us for 8
// rows of 8 of 64 experts (K = 2048, N_out = 1408, 7.3 MB). What bounds the
// latter: every CTA quantizes all 8 rows, and codes, keep bits, selectors,
// activations and partial sums all pass through shared memory (stalls on its
// pipe come first; 47 % of the issue slots taken, DRAM 6 % busy).
#pragma once

#include "async.cuh"
#include "bl_gemv.cuh"
#include "common.cuh"
#include "epi.cuh"
#include "grp.cuh"

namespace sbn {

constexpr int kGgMaxRows = 16;
constexpr int kGgMaxSlots = 16;
// Arrival barriers, taken in turn by the tiles of a CTA (tile % kGgArrivals,
// whatever its slot). A wait by parity for tile t must not meet a barrier whose
// earlier tile t - kGgArrivals is still to come. A warp's tiles lie at most 31
// apart (items are dealt out to 31 warps), and a tile that has landed was
// issued, so every tile a ring before it had been consumed: with at least 31 +
// slots barriers, t - kGgArrivals is one of those. One barrier per slot let
// warps that start two rounds ahead (K <= 256) pass before any copy had landed.
constexpr int kGgArrivals = 48;
static_assert(kGgArrivals >= kGvConsumerWarps + kGgMaxSlots, "no wait by parity may be two phases off");

struct GgLayout {
  uint32_t sel, list, rmax, scale, mult, full, empty, cnt, acc, x, codes, meta, total;
  int xstride, slots;
};

// Shared-memory layout with as many slots as fit (at most `tiles` and
// kGgMaxSlots); slots = 0 if not even two fit (one, for a single tile).
__host__ __device__ inline GgLayout gg_layout(int tiles, int nt, int t, int k, int cstride, int mstride) {
  GgLayout L;
  L.xstride = k + 16;
  const int want = tiles < kGgMaxSlots ? tiles : kGgMaxSlots;
  for (L.slots = want; L.slots > 0; --L.slots) {
    const int S = L.slots;
    L.sel = 0;                                   // 256 selector pairs
    L.list = 2048;                               // header (count) and 16 entries of 16 bytes
    L.rmax = L.list + 16 + kGgMaxRows * 16;      // row maxima, scales, multipliers
    L.scale = L.rmax + kGgMaxRows * 4;
    L.mult = L.scale + kGgMaxRows * 4;
    L.full = gv_align128(L.mult + kGgMaxRows * 4);
    L.empty = L.full + 8 * kGgArrivals;
    L.cnt = L.empty + 8 * S;
    L.acc = gv_align128(L.cnt + 4 * S);          // [S][16][nt] int32
    L.x = gv_align128(L.acc + (size_t)S * 16 * nt * 4);
    L.codes = gv_align128(L.x + (size_t)t * L.xstride);
    L.meta = gv_align128(L.codes + (size_t)S * 16 * cstride);
    const size_t total = L.meta + (size_t)S * 16 * mstride;
    if (total <= kGvSmemMax) {
      L.total = (uint32_t)total;
      if (S >= 2 || tiles == 1) return L;
      break;
    }
  }
  L.slots = 0;
  L.total = 0;
  return L;
}

struct GgParams {
  const int8_t* xq;       // INT8 activations [R, K] and scales [R] (not XBF)
  const float* xs;
  const uint16_t* xbf;    // XBF: bf16 activations [R, K]
  int8_t* xq_out;         // XBF: optional copies of Xq and s (written by CTA 0)
  float* xs_out;
  const uint8_t* codes;   // [E, N_out, cstride]
  const uint8_t* meta;
  const float* gamma;     // [E]
  uint16_t* y;
  EpiParams ep;
  GrpParams grp;
  int K, N;
  int cstride, mstride;
  int kc;                 // 16-byte activation chunks per row (K/8 bf16 or K/16 INT8)
  uint32_t kc_magic;      // ceil(2^32 / kc)
  int dr, drem;           // 992 = dr * kc + drem
  GgLayout L;
};

template <int MM, int CB, int NT, bool DENSE, bool XBF>
__global__ void __launch_bounds__(kGvThreads, 1)
bl_gemv_grp_kernel(const GgParams p) {
  extern __shared__ __align__(128) uint8_t gg_smem[];
  const GgLayout& L = p.L;
  const int S = L.slots, R = p.grp.rows;
  uint2* s_sel2 = reinterpret_cast<uint2*>(gg_smem + L.sel);
  int* s_head = reinterpret_cast<int*>(gg_smem + L.list);              // [0]: experts with rows
  int4* s_list = reinterpret_cast<int4*>(gg_smem + L.list + 16);       // first row, rows, expert, gamma
  uint32_t* s_rmax = reinterpret_cast<uint32_t*>(gg_smem + L.rmax);
  float* s_scale = reinterpret_cast<float*>(gg_smem + L.scale);
  float* s_mult = reinterpret_cast<float*>(gg_smem + L.mult);
  uint64_t* s_full = reinterpret_cast<uint64_t*>(gg_smem + L.full);
  uint64_t* s_empty = reinterpret_cast<uint64_t*>(gg_smem + L.empty);
  int* s_cnt = reinterpret_cast<int*>(gg_smem + L.cnt);
  int32_t* s_acc = reinterpret_cast<int32_t*>(gg_smem + L.acc);
  uint8_t* s_x = gg_smem + L.x;
  uint8_t* s_codes = gg_smem + L.codes;
  uint8_t* s_meta = gg_smem + L.meta;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tpe = (p.N + 15) / 16;   // tiles per expert
  const int ipt = (p.K + 255) / 256;  // items per tile

  // this CTA's range [begin, begin + tiles) of the work list
  auto range = [&](int active, int& begin) {
    const int total = active * tpe, base = total / (int)gridDim.x, rem = total % (int)gridDim.x;
    const int bid = (int)blockIdx.x;
    begin = bid * base + min(bid, rem);
    return base + (bid < rem ? 1 : 0);
  };

  if (warp == kGvConsumerWarps) {
    // ---- producer warp ----
    if (lane < kGgMaxRows) s_rmax[lane] = 0u;
    for (int i = lane; i < kGgArrivals; i += 32) mbar_init(&s_full[i], 1);
    if (lane < S) {
      mbar_init(&s_empty[lane], 1);
      s_cnt[lane] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    griddep_wait();
    int active = 0;
    if (p.grp.offsets == nullptr) {
      active = 1;
      if (lane == 0) s_list[0] = make_int4(0, R, 0, __float_as_int(__ldg(p.gamma)));
    } else {
      // experts e0 + lane, four groups of 32 offsets in flight at a time
      const int E = p.grp.experts;
      int top = 0;
      for (int e00 = 0; e00 < E; e00 += 128) {
        int v[4], nx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = e00 + 32 * j + lane;
          v[j] = e <= E ? p.grp.offsets[e] : 0;
          nx[j] = e00 + 32 * j + 32 <= E ? p.grp.offsets[e00 + 32 * j + 32] : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = e00 + 32 * j + lane;
          int lo = min(max(v[j], 0), R);
          lo = max(warp_scan_max(lo, lane), top);
          top = __shfl_sync(0xffffffffu, lo, 31);
          int hi = __shfl_down_sync(0xffffffffu, lo, 1);
          if (lane == 31) hi = max(top, min(max(nx[j], 0), R));
          const bool on = e < E && hi > lo;
          const uint32_t b = __ballot_sync(0xffffffffu, on);
          const int at = active + __popc(b & ((1u << lane) - 1u));
          if (on && at < kGgMaxRows) s_list[at] = make_int4(lo, hi - lo, e, __float_as_int(__ldg(p.gamma + e)));
          active += __popc(b);
        }
      }
      active = min(active, kGgMaxRows);   // non-empty and disjoint: at most R of them
    }
    if (lane == 0) s_head[0] = active;
    __syncwarp();
    gv_setup_arrive();
    int begin;
    const int tiles = range(active, begin);
    if (lane == 0) {
      for (int i = 0; i < tiles; ++i) {
        const int slot = i % S;
        if (i >= S && !mbar_wait(&s_empty[slot], ((i / S) & 1u) ^ 1u)) break;
        const int a = (begin + i) / tpe, r = ((begin + i) - a * tpe) * 16;
        const size_t row = (size_t)s_list[a].z * p.N + r;
        const uint32_t rows = (uint32_t)min(16, p.N - r);
        const uint32_t cbytes = rows * (uint32_t)p.cstride;
        const uint32_t mbytes = DENSE ? 0u : rows * (uint32_t)p.mstride;
        uint64_t* full = &s_full[i % kGgArrivals];
        mbar_arrive_expect_tx(full, cbytes + mbytes);
        bulk_g2s(s_codes + (size_t)slot * 16 * p.cstride, p.codes + row * p.cstride, cbytes, full);
        if (!DENSE) bulk_g2s(s_meta + (size_t)slot * 16 * p.mstride, p.meta + row * p.mstride, mbytes, full);
      }
    }
    return;   // every copy is waited for by the consumers before they leave
  }

  // ---- consumers: activations global -> registers (bl_gemv.cuh) ----
  griddep_wait();
  const int kc = p.kc, nq = R * kc;
  const bool xwarp = warp * 32 < nq;
  const int q0r = (int)__umulhi((uint32_t)tid, p.kc_magic);
  const int q0c = tid - q0r * kc;
  const uint4* xsrc = reinterpret_cast<const uint4*>(XBF ? static_cast<const void*>(p.xbf)
                                                         : static_cast<const void*>(p.xq));
  uint4 v[kGvMaxChunks];
  if (xwarp) {
#pragma unroll
    for (int j = 0; j < kGvMaxChunks; ++j) {
      const int q = tid + j * kGvConsumers;
      if (q < nq) v[j] = __ldg(xsrc + q);
    }
  }
  if (!XBF && tid < R) s_scale[tid] = __ldg(p.xs + tid);
  if (!DENSE && tid < 256) s_sel2[tid] = gv_selector_pair((uint32_t)tid);
  for (int i = tid; i < S * 16 * NT; i += kGvConsumers) s_acc[i] = 0;
  gv_setup_wait();   // list, barriers and row maxima are written

  if (XBF) {
    if (xwarp) {
      int r = q0r, c = q0c;
#pragma unroll
      for (int j = 0; j < kGvMaxChunks; ++j) {
        if (j * kGvConsumers + warp * 32 >= nq) break;
        const bool ok = tid + j * kGvConsumers < nq;
        const uint32_t m2 = ok ? gv_chunk_absmax(v[j], 0u) : 0u;
        const uint32_t m = ok ? max(m2 & 0x7FFFu, (m2 >> 16) & 0x7FFFu) : 0u;
        const int row = ok ? r : -1;
        uint32_t todo = __ballot_sync(0xffffffffu, ok);
        while (todo) {
          const int lead = __ffs(todo) - 1;
          const int lr = __shfl_sync(0xffffffffu, row, lead);
          const bool mine = row == lr;
          const uint32_t rm = __reduce_max_sync(0xffffffffu, mine ? m : 0u);
          if (lane == lead) atomicMax(&s_rmax[lr], rm);
          todo &= ~__ballot_sync(0xffffffffu, mine);
        }
        r += p.dr;
        c += p.drem;
        if (c >= kc) { c -= kc; ++r; }
      }
    }
    gv_consumer_sync();
    if (tid < R) {
      const float sc = fmaxf(__uint_as_float(s_rmax[tid] << 16), 1e-5f);
      s_mult[tid] = __fdiv_rn(127.0f, sc);
      s_scale[tid] = sc;
      if (blockIdx.x == 0 && p.xs_out) p.xs_out[tid] = sc;
    }
    gv_consumer_sync();
  }
  if (xwarp) {
    const bool out = XBF && blockIdx.x == 0 && p.xq_out != nullptr;
    int r = q0r, c = q0c;
#pragma unroll
    for (int j = 0; j < kGvMaxChunks; ++j) {
      if (j * kGvConsumers + warp * 32 >= nq) break;
      if (tid + j * kGvConsumers < nq) {
        if (XBF) {
          const uint2 q = quant8_magic(v[j], s_mult[r]);
          *reinterpret_cast<uint2*>(s_x + (size_t)r * L.xstride + gv_xchunk(c >> 1) + 8 * (c & 1)) = q;
          if (out) *reinterpret_cast<uint2*>(p.xq_out + (size_t)r * p.K + 8 * (size_t)c) = q;
        } else {
          *reinterpret_cast<uint4*>(s_x + (size_t)r * L.xstride + gv_xchunk(c)) = v[j];
        }
      }
      r += p.dr;
      c += p.drem;
      if (c >= kc) { c -= kc; ++r; }
    }
  }
  gv_consumer_sync();

  // ---- contraction ----
  const int g = lane >> 2, t = lane & 3;
  int begin;
  const int tiles = range(s_head[0], begin);
  const int items = tiles * ipt;
  for (int it = warp; it < items; it += kGvConsumerWarps) {
    const int tile = it / ipt, kit = it - tile * ipt;
    const int slot = tile % S;
    const int a = (begin + tile) / tpe;
    const int r0 = ((begin + tile) - a * tpe) * 16;   // first weight row of the tile
    const int4 ex = s_list[a];
    const int row0 = ex.x, nrow = ex.y;
    if (!mbar_wait_warp(&s_full[tile % kGgArrivals], (tile / kGgArrivals) & 1u)) break;
    const int span = kit * 256 + 64 * t;   // first position of this thread's 64
    const bool valid = span < p.K;
    uint32_t cw[2][CB];
    uint32_t mw[2][2];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int r = slot * 16 + g + 8 * rr;
      const uint32_t* cp = reinterpret_cast<const uint32_t*>(s_codes + (size_t)r * p.cstride + span / 16 * CB);
#pragma unroll
      for (int j = 0; j < CB; ++j) cw[rr][j] = valid ? cp[j] : 0u;
      mw[rr][0] = mw[rr][1] = 0u;
      if (!DENSE && valid) {
        const uint2 m = *reinterpret_cast<const uint2*>(s_meta + (size_t)r * p.mstride + span / 8);
        mw[rr][0] = m.x;
        mw[rr][1] = m.y;
      }
    }
    const uint8_t* xa = s_x + (size_t)(row0 + g) * L.xstride;
    const uint8_t* xb = s_x + (size_t)(row0 + g + 8) * L.xstride;
    const bool la = valid && g < nrow, lb = valid && NT == 16 && g + 8 < nrow;
    int acc0[4] = {0, 0, 0, 0};
    int acc1[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int xo = gv_xchunk(span / 16 + j);
      const uint4 fa = la ? *reinterpret_cast<const uint4*>(xa + xo) : make_uint4(0u, 0u, 0u, 0u);
      uint4 fb = make_uint4(0u, 0u, 0u, 0u);
      if (NT == 16) fb = lb ? *reinterpret_cast<const uint4*>(xb + xo) : fb;
      uint32_t a00, a01, a10, a11, b00, b01, b10, b11;
#define SBN_GG_PAIR(IA, IB)                                     \
      gv_expand<MM, CB, DENSE, IA>(cw[0], mw[0], s_sel2, a00, a01); \
      gv_expand<MM, CB, DENSE, IA>(cw[1], mw[1], s_sel2, a10, a11); \
      gv_expand<MM, CB, DENSE, IB>(cw[0], mw[0], s_sel2, b00, b01); \
      gv_expand<MM, CB, DENSE, IB>(cw[1], mw[1], s_sel2, b10, b11);
      if (j == 0) {
        SBN_GG_PAIR(0, 1)
      } else if (j == 1) {
        SBN_GG_PAIR(2, 3)
      } else if (j == 2) {
        SBN_GG_PAIR(4, 5)
      } else {
        SBN_GG_PAIR(6, 7)
      }
#undef SBN_GG_PAIR
      mma_s8_16x8x32(acc0, a00, a10, a01, a11, fa.x, fa.y);
      mma_s8_16x8x32(acc0, b00, b10, b01, b11, fa.z, fa.w);
      if (NT == 16) {
        mma_s8_16x8x32(acc1, a00, a10, a01, a11, fb.x, fb.y);
        mma_s8_16x8x32(acc1, b00, b10, b01, b11, fb.z, fb.w);
      }
    }
    int32_t* acc = s_acc + (size_t)slot * 16 * NT;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (2 * t + j < nrow) {
        atomicAdd(&acc[g * NT + 2 * t + j], acc0[j]);
        atomicAdd(&acc[(g + 8) * NT + 2 * t + j], acc0[2 + j]);
      }
      if (NT == 16 && 8 + 2 * t + j < nrow) {
        atomicAdd(&acc[g * NT + 8 + 2 * t + j], acc1[j]);
        atomicAdd(&acc[(g + 8) * NT + 8 + 2 * t + j], acc1[2 + j]);
      }
    }
    __syncwarp();
    int last = 0;
    if (lane == 0) {
      __threadfence_block();   // the warp's sums before its count
      last = atomicAdd(&s_cnt[slot], 1) == ipt - 1;
      __threadfence_block();
    }
    if (!__shfl_sync(0xffffffffu, last, 0)) continue;
    __syncwarp();   // the other warps' sums, which lane 0 has seen counted, before every lane's reads
    // ---- epilogue of the tile: 16 outputs of every row of the expert ----
    const float gm = __int_as_float(ex.w);
    for (int i = lane; i < 16 * nrow; i += 32) {
      const int r = i & 15, row = row0 + (i >> 4), o = r0 + r;
      int32_t* ap = acc + r * NT + (i >> 4);
      const int av = *ap;
      *ap = 0;
      if (o < p.N) {
        const size_t at = (size_t)row * p.N + o;
        const float bias = p.ep.bias ? __ldg(p.ep.bias + (size_t)ex.z * p.N + o) : 0.f;
        const float z = __fmaf_rn((float)av, __fdiv_rn(__fmul_rn(gm, s_scale[row]), 127.0f), bias);
        if (p.ep.z) p.ep.z[at] = f32_to_bf16_bits(z);
        float yv = act_f(p.ep.act, z);
        if (p.ep.residual) yv = __fadd_rn(yv, bf16_bits_to_float(p.ep.residual[at]));
        p.y[at] = f32_to_bf16_bits(yv);
      }
    }
    if (lane == 0) s_cnt[slot] = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&s_empty[slot]);
  }
  griddep_launch_dependents();
}

}  // namespace sbn
