// The epilogue of one warp of a tensor-core kernel: chunks of 32 output
// features (TMEM lanes) x 32 tokens (columns) of int32 accumulators.
//
// The accumulators are read in the 16 x 256-bit shape, which gives a thread
// two neighbouring tokens of a feature: the fragments of 8 x 8 matrices, so
// that stmatrix.trans writes the packed bf16 pairs token by token (4
// instructions for a chunk; one 2-byte store per element, from the shape that
// gives a thread one feature's row, made the epilogue half of the kernel's
// instructions). Where every output row starts on a 16-byte boundary, a chunk
// goes through a 2 KB tile of shared memory, 64 bytes per token, 64-byte
// swizzle: the residual is read with one 64-byte run per token (lane = token)
// into the tile and taken up with ldmatrix.trans, and the tile leaves with
// one TMA store. A chunk that ends inside the tile of another expert's rows
// (tok_end) is written with 16-byte stores of its own tokens instead: the
// rows behind belong to someone else. Other outputs are written element by
// element.
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

// Byte offset of 16-byte piece c (8 features) of a token's row in the tile.
SBN_DEVFN uint32_t epi_piece(int token, int c) { return (uint32_t)(token * 64 + ((c ^ ((token >> 1) & 3)) << 4)); }

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
    uint4* d = reinterpret_cast<uint4*>(dst + (size_t)(tok + lane) * N + row_w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row_w + 8 * i < N)
        d[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(tile) + epi_piece(lane, i));
  }
}

// 16 lanes x 32 columns. Registers 4 i .. 4 i + 3 of a thread: columns 8 i + 2
// (lane % 4) and the next one, of lane lane / 4 and of lane lane / 4 + 8. Load
// and wait in one statement: between the two the registers must not be
// touched, and a compiler may well copy them there.
SBN_DEVFN void tmem_ld16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
SBN_DEVFN void st_matrix4_trans(uint32_t addr, const uint32_t* p) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(p[0]),
               "r"(p[1]), "r"(p[2]), "r"(p[3])
               : "memory");
}
SBN_DEVFN void ld_matrix4_trans(uint32_t addr, uint32_t* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
               : "r"(addr)
               : "memory");
}
// Two fp32 -> a bf16 pair, a in the low half.
SBN_DEVFN uint32_t pack_bf16(float a, float b) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

// One chunk, in two halves of 16 features. taddr: the chunk's accumulators
// (feature row_w + lane, tokens tok .. tok + 31); sc: gamma s / 127 of token
// tok + lane; bias: of feature row_w + lane. res is this chunk's residual and
// is reloaded for the next one (next_tok < 0: none). done, if not NULL, is
// arrived on once per warp as soon as the accumulators are in registers.
SBN_DEVFN void epi_chunk(const EpiParams& ep, const EpiOut& o, EpiTile& t, uint32_t taddr, float sc, float bias,
                         int row_w, int tok, int tok_end, int next_tok, int lane, uint4 (&res)[4], uint64_t* done) {
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
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(yb) + epi_piece(lane, i)) = res[i];
      if (next_tok >= 0) epi_load_residual(ep, o, row_w, next_tok, tok_end, lane, res);
    }
  }
  __syncwarp();
  const int c2 = 2 * (lane & 3), fr = lane >> 2;   // the thread's tokens 8 i + c2, + 1; features fr, fr + 8 of a half
  // its row of the matrices of two token groups: token 8 ((lane >> 4) & 1) + lane % 8, piece (lane >> 3) & 1
  const int mt = ((lane >> 4) << 3) + (lane & 7), mp = (lane >> 3) & 1;
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = *reinterpret_cast<const float2*>(t.sc + 8 * i + c2);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r[16];
    tmem_ld16x32(taddr + ((uint32_t)(16 * h) << 16), r);
    if (h == 1 && done) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(done);
    }
    const float b0 = __shfl_sync(0xffffffffu, bias, 16 * h + fr), b1 = __shfl_sync(0xffffffffu, bias, 16 * h + fr + 8);
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = __fmaf_rn((float)(int32_t)r[4 * i], f[i].x, b0);
      v[4 * i + 1] = __fmaf_rn((float)(int32_t)r[4 * i + 1], f[i].y, b0);
      v[4 * i + 2] = __fmaf_rn((float)(int32_t)r[4 * i + 2], f[i].x, b1);
      v[4 * i + 3] = __fmaf_rn((float)(int32_t)r[4 * i + 3], f[i].y, b1);
    }
    if (o.aligned) {
      // addresses of the matrices (token groups 2 k and 2 k + 1)
      const uint32_t at[2] = {epi_piece(mt, 2 * h + mp), epi_piece(16 + mt, 2 * h + mp)};
      uint32_t p[8];
      if (ep.z) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        st_matrix4_trans(smem_u32(zb) + at[0], p);
        st_matrix4_trans(smem_u32(zb) + at[1], p + 4);
      }
      act_all(ep.act, v);
      if (ep.residual) {
        ld_matrix4_trans(smem_u32(yb) + at[0], p);
        ld_matrix4_trans(smem_u32(yb) + at[1], p + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[2 * i] = __fadd_rn(v[2 * i], __uint_as_float(p[i] << 16));
          v[2 * i + 1] = __fadd_rn(v[2 * i + 1], __uint_as_float(p[i] & 0xFFFF0000u));
        }
        __syncwarp();   // the half's residual is read before it is overwritten
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      st_matrix4_trans(smem_u32(yb) + at[0], p);
      st_matrix4_trans(smem_u32(yb) + at[1], p + 4);
    } else {
      const int row = row_w + 16 * h + fr;
      float u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = v[i];
      act_all(ep.act, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int tk = tok + 8 * (i >> 2) + c2 + (i & 1), rw = row + ((i & 2) ? 8 : 0);
        if (rw < o.N && tk < tok_end) {
          const size_t at = (size_t)tk * o.N + rw;
          if (ep.z) ep.z[at] = f32_to_bf16_bits(u[i]);
          if (ep.residual) v[i] = __fadd_rn(v[i], bf16_bits_to_float(ep.residual[at]));
          o.y[at] = f32_to_bf16_bits(v[i]);
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
