// Backward of the layer's epilogue: dz = dy f'(z) and the bias gradient, the
// column sums of dz (per expert where the rows are grouped).
//
// Bound by DRAM: dy and z are read and dz is written once, 6 bytes per
// element. A cluster of CTAs owns 64 columns of one expert's rows: 8 lanes of
// eight columns (16-byte accesses, a 128-byte line per row) by 32 row lanes
// per CTA. The column sums stay in registers (fp32, of the unrounded dz), then
// go through shared memory and the cluster's distributed shared memory in a
// fixed order: no workspace, no atomics, the same sums every time. The
// cluster is as small (1, 2, 4 or 8 CTAs) as fills the GPU: the CTAs of a
// cluster start and end together, and with eight of them per block of columns a
// batch over 16 experts ran at a third of the bandwidth. Where N_out is not a
// multiple of 8 a lane takes every 8th column with 2-byte accesses.
// Measured at 4096 rows of 6912 features, 16 experts: 31 to 34 us, 5.0 to 5.5
// TB/s, 78 to 85 % of the copy rate; at 509 rows the kernel takes 9 us, the call
// 13.3. 6911 features, by 2-byte accesses: 59 us where 6912 take 29 (captured
// calls, one after the other).
#pragma once

#include "common.cuh"
#include "epi.cuh"
#include "grp.cuh"
#include "pair.cuh"

namespace sbn {

constexpr int kAgThreads = 256;
constexpr int kAgCols = 64;        // columns per cluster
constexpr int kAgColLanes = 8;
constexpr int kAgLanes = kAgThreads / kAgColLanes;   // row lanes per CTA
constexpr int kAgUnroll = 4;       // rows of a lane in flight

struct AgParams {
  const uint16_t* dy;
  const uint16_t* z;
  uint16_t* dz;    // may be dy: a thread reads its elements before it writes them
  float* dbias;     // [E, N] or NULL
  GrpParams grp;
  int N;
  int act;
  int cluster;      // CTAs per cluster
};

// Grid (column blocks x cluster, experts).
template <bool VEC>
__global__ void __launch_bounds__(kAgThreads)
act_grad_kernel(const AgParams p) {
  __shared__ float s_sum[kAgLanes][kAgCols];
  __shared__ float s_cta[kAgCols];
  const int tid = threadIdx.x, lane_r = tid / kAgColLanes, lane_c = tid % kAgColLanes;
  const int cs = p.cluster;
  const int rank = (int)(blockIdx.x % (unsigned)cs);
  const int c0 = (int)(blockIdx.x / (unsigned)cs) * kAgCols;
  const int e = (int)blockIdx.y;
  griddep_wait();
  int lo = 0, hi = p.grp.rows;
  if (p.grp.offsets) {
    // as grp_build has them: the largest offset so far, so that no row belongs
    // to two experts whatever the offsets are (every warp for itself, which saves
    // a barrier: 31 to 34 us at 4096 rows of 16 experts, 31 to 36 with one)
    const int next = p.grp.offsets[e + 1];
    int top = 0;
    for (int i = tid & 31; i <= e; i += 32) top = max(top, p.grp.offsets[i]);
    top = __reduce_max_sync(0xffffffffu, top);
    lo = min(top, p.grp.rows);
    hi = min(max(next, lo), p.grp.rows);
  }
  const int step = VEC ? 1 : kAgColLanes;   // distance between a lane's columns
  const int col = c0 + (VEC ? 8 * lane_c : lane_c);
  float sum[8] = {};
  // unsigned: up to kAgUnroll * cs * kAgLanes past the last row, which may be the 2^31st
  const unsigned end = (unsigned)hi, stride = (unsigned)(cs * kAgLanes);
  for (unsigned r0 = (unsigned)lo + (unsigned)(rank * kAgLanes + lane_r); r0 < end; r0 += kAgUnroll * stride) {
    uint4 dv[kAgUnroll], zv[kAgUnroll];
    float d[8], z[8];
    if (VEC) {
#pragma unroll
      for (int u = 0; u < kAgUnroll; ++u) {
        const unsigned r = r0 + u * stride;
        if (r < end && col < p.N) {
          dv[u] = *reinterpret_cast<const uint4*>(p.dy + (size_t)r * p.N + col);
          zv[u] = *reinterpret_cast<const uint4*>(p.z + (size_t)r * p.N + col);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAgUnroll; ++u) {
      const unsigned r = r0 + u * stride;
      if (r >= end || col >= p.N) continue;
      const size_t at = (size_t)r * p.N + col;
      if (VEC) {
        const uint32_t dw[4] = {dv[u].x, dv[u].y, dv[u].z, dv[u].w}, zw[4] = {zv[u].x, zv[u].y, zv[u].z, zv[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[2 * j] = __uint_as_float(dw[j] << 16);
          d[2 * j + 1] = __uint_as_float(dw[j] & 0xFFFF0000u);
          z[2 * j] = __uint_as_float(zw[j] << 16);
          z[2 * j + 1] = __uint_as_float(zw[j] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool ok = col + j * step < p.N;
          d[j] = ok ? bf16_bits_to_float(p.dy[at + j * step]) : 0.f;
          z[j] = ok ? bf16_bits_to_float(p.z[at + j * step]) : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] *= act_df(p.act, z[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += d[j];
      if (VEC) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = (uint32_t)f32_to_bf16_bits(d[2 * j]) | ((uint32_t)f32_to_bf16_bits(d[2 * j + 1]) << 16);
        *reinterpret_cast<uint4*>(p.dz + at) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j * step < p.N) p.dz[at + j * step] = f32_to_bf16_bits(d[j]);
      }
    }
  }
  griddep_launch_dependents();
  if (!p.dbias) return;   // the same for every CTA of the cluster
#pragma unroll
  for (int j = 0; j < 8; ++j) s_sum[lane_r][col - c0 + j * step] = sum[j];
  __syncthreads();
  if (tid < kAgCols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kAgLanes; ++i) t += s_sum[i][tid];
    s_cta[tid] = t;
    if (cs == 1 && c0 + tid < p.N) p.dbias[(size_t)e * p.N + c0 + tid] = t;
  }
  if (cs == 1) return;
  cluster_sync_all();
  if (rank == 0 && tid < kAgCols && c0 + tid < p.N) {
    float t = 0.f;
    for (int c = 0; c < cs; ++c) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_rank(smem_u32(&s_cta[tid]), (uint32_t)c)));
      t += v;
    }
    p.dbias[(size_t)e * p.N + c0 + tid] = t;
  }
  cluster_sync_all();   // no CTA leaves while its sums are read
}

}  // namespace sbn
