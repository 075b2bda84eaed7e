// The epilogue of one warp of a tensor-core kernel: chunks of 32 output
// features (TMEM lanes) x 32 tokens (columns) of int32 accumulators.
//
// Where every output row starts on a 16-byte boundary, a chunk goes through a
// 2 KB tile of shared memory [token][feature]: the residual is read with one
// 64-byte run per token (lane = token) into the tile, each lane then works down its feature's
// column in place, and the tile leaves with one TMA store. A chunk that ends
// inside the tile of another expert's rows (tok_end) is written with 16-byte
// stores of its own tokens instead: the rows behind belong to someone else.
// Other outputs are written element by element.
#pragma once

#include <cuda.h>

#include "epi.cuh"
#include "pair.cuh"

namespace sbn {

struct EpiTile {
  uint16_t* buf;     // this warp's two 32 x 32 tiles
  float* sc;         // and 32 floats
  int nstore;        // TMA stores so far (the tile to use next without z)
};

struct EpiOut {
  const CUtensorMap* ty;   // 32 x 32 boxes of y and z (aligned only)
  const CUtensorMap* tz;
  uint16_t* y;
  int N;
  int rows;          // rows of the whole output (the TMA store ends there)
  bool aligned;      // 16-byte rows of y, z and the residual
};

SBN_DEVFN void tma_store_wait_read0() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }

// The residual of a chunk: lane's token, 32 features from row_w on.
SBN_DEVFN void epi_load_residual(const EpiParams& ep, const EpiOut& o, int row_w, int tok, int tok_end, int lane,
                                 uint4 (&res)[4]) {
  if (!ep.residual || !o.aligned) return;
  const bool ok = tok + lane < tok_end;
  const uint4* src = reinterpret_cast<const uint4*>(ep.residual + (size_t)(tok + lane) * o.N + row_w);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    res[i] = (ok && row_w + 8 * i < o.N) ? src[i] : make_uint4(0u, 0u, 0u, 0u);
}

// 16-byte stores of the tokens below tok_end of a staged tile.
SBN_DEVFN void epi_store_rows(uint16_t* dst, const uint16_t* tile, int N, int row_w, int tok, int tok_end, int lane) {
  if (tok + lane < tok_end) {
    const uint4* src = reinterpret_cast<const uint4*>(tile + lane * 32);
    uint4* d = reinterpret_cast<uint4*>(dst + (size_t)(tok + lane) * N + row_w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row_w + 8 * i < N) d[i] = src[i];
  }
}

// 16 columns of this warp's 32 lanes. Load and wait in one statement: between
// the two the registers must not be touched, and a compiler may well copy
// them there when they live across a loop's edge.
SBN_DEVFN void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// One chunk, sixteen tokens at a time in a rolled loop: unrolled over all 32,
// its code and the producers' kept evicting each other from the instruction
// cache. taddr: the chunk's accumulators (feature row_w + lane, tokens tok ..
// tok + 31); sc: gamma s / 127 of token tok + lane; bias: of the lane's
// feature. res is this chunk's residual and is reloaded for the next one
// (next_tok < 0: none).
SBN_DEVFN void epi_chunk(const EpiParams& ep, const EpiOut& o, EpiTile& t, uint32_t taddr, float sc, float bias,
                         int row_w, int tok, int tok_end, int next_tok, int lane, uint4 (&res)[4]) {
  const int row = row_w + lane;
  const bool whole = tok + 32 <= tok_end || tok_end == o.rows;
  const bool inside = row_w < o.N && tok < tok_end;
  uint16_t* zb = t.buf;
  uint16_t* yb = t.buf + (ep.z ? 1024 : (t.nstore & 1) * 1024);
  __syncwarp();   // the previous chunk's reads of the factors are done
  t.sc[lane] = sc;
  if (o.aligned) {
    if (lane == 0) {
      if (ep.z) tma_store_wait_read0();
      else tma_store_wait_read1();
    }
    __syncwarp();
    if (ep.residual) {
      uint4* d = reinterpret_cast<uint4*>(yb + lane * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = res[i];
      if (next_tok >= 0) epi_load_residual(ep, o, row_w, next_tok, tok_end, lane, res);
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t r[16];
    tmem_ld16(taddr + 16u * (uint32_t)h, r);
    // the tokens' factors by 16-byte broadcast reads (a shuffle per element
    // cost as much as the rest of a plain epilogue)
    float v[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 f = reinterpret_cast<const float4*>(t.sc)[4 * h + j];
      v[4 * j] = __fmaf_rn((float)(int32_t)r[4 * j], f.x, bias);
      v[4 * j + 1] = __fmaf_rn((float)(int32_t)r[4 * j + 1], f.y, bias);
      v[4 * j + 2] = __fmaf_rn((float)(int32_t)r[4 * j + 2], f.z, bias);
      v[4 * j + 3] = __fmaf_rn((float)(int32_t)r[4 * j + 3], f.w, bias);
    }
    if (o.aligned) {
      const int at = 512 * h + lane;
      if (ep.z) {
#pragma unroll
        for (int j = 0; j < 16; ++j) zb[at + 32 * j] = f32_to_bf16_bits(v[j]);
      }
      act_all(ep.act, v);
      if (ep.residual) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __fadd_rn(v[j], bf16_bits_to_float(yb[at + 32 * j]));
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) yb[at + 32 * j] = f32_to_bf16_bits(v[j]);
    } else {
      const int tk = tok + 16 * h;
      const size_t at = (size_t)tk * o.N + row;
      if (ep.z) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (row < o.N && tk + j < tok_end) ep.z[at + (size_t)j * o.N] = f32_to_bf16_bits(v[j]);
      }
      act_all(ep.act, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (row < o.N && tk + j < tok_end) {
          if (ep.residual) v[j] = __fadd_rn(v[j], bf16_bits_to_float(ep.residual[at + (size_t)j * o.N]));
          o.y[at + (size_t)j * o.N] = f32_to_bf16_bits(v[j]);
        }
      }
    }
  }
  if (!o.aligned) return;
  if (whole) asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  __syncwarp();
  if (!inside) return;
  if (whole) {
    if (lane == 0) {
      if (ep.z) tma_store_2d(o.tz, row_w, tok, zb);
      tma_store_2d(o.ty, row_w, tok, yb);
    }
    ++t.nstore;
  } else {
    if (ep.z) epi_store_rows(ep.z, zb, o.N, row_w, tok, tok_end, lane);
    epi_store_rows(o.y, yb, o.N, row_w, tok, tok_end, lane);
  }
}

}  // namespace sbn
