// AdamW over many tensors in one launch, states in 32 or in 8 bits.
//
// The latent weights of a ternary layer take their gradients in full
// precision ("BitNet b1.58: How Ternary Weights Cut LLM Memory by 82% Without
// Losing Accuracy", section "How ternary quantization works during
// training"); Sparse-BitNet trains them with AdamW (Table 5: betas 0.9 and
// 0.95, decoupled weight decay). With t = step + 1, per element
//     m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// every product and sum rounded on its own in fp32 (no fused multiply-add),
// so that an elementwise evaluation gives the same bits of m and v. p's quotient
// goes through an approximate reciprocal and the bias corrections through
// expm1f: p is within 32 half steps of its update.
//
// 8-bit states: a block of 256 elements shares one power of two per state;
// m and r = sqrt(v) are held as e4m3 codes times it. The codes round up with
// the probability of the remainder (a hash of seed, step, tensor and index
// gives the random bits): with rounding to nearest, v would never move, since
// one step changes it by at most 1 - b2 of itself, less than half a code. r
// rather than v is held because its range is half as many binades; a
// positive r never becomes code 0, so a denominator cannot vanish. What is not
// finite becomes the NaN code (e4m3 has no infinity) and does not count for the
// block's scale, so its neighbours keep their codes.
//
// One warp owns a block of 256 elements, eight to a lane (256-bit accesses of
// fp32, 128-bit of bf16, 64-bit of codes), the persistent CTAs stride over
// the segments of 2048 elements of all tensors. The tensor table is a kernel
// parameter: no copy to the device, nothing to keep alive, and the call can be
// captured into a graph. 28 bytes per element with an fp32 master, its bf16 copy
// and fp32 states, 16 with 8-bit states. Measured at 114 million elements (72
// tensors): 32-bit states 559 us, 5.7 TB/s, 89 % of the copy rate, bound by DRAM;
// 8-bit states 462 us, 4.0 TB/s, 61 %, bound by instruction issue (74 % of the
// slots, about 100 instructions per element: the two roundings, the hash and the
// blocks' maxima). With bf16 parameters 438 and 488 us: there the 8-bit states
// save memory, not time. A step of 24 small tensors takes 6.6 us on the device.
#pragma once

#include "common.cuh"

namespace sbn {

constexpr int kAwThreads = 256;
constexpr int kAwBlock = 256;                        // elements per warp step and 8-bit scale
constexpr int kAwSeg = kAwBlock * (kAwThreads / 32);  // elements per CTA step
constexpr uint32_t kAwHashA = 0x9E3779B1u, kAwHashB = 0xB7E15163u;

struct AwEntry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  uint32_t numel;
  uint32_t vec;   // every array aligned for the wide accesses
};

template <int N>
struct AwTable {
  AwEntry e[N];
  uint32_t first[N + 1];   // segments before tensor i
  int count;
  uint32_t id0;            // index of the first tensor in the whole call (hash)
  int last;                // this launch advances the step
};

struct AwHyper {
  int* step;
  const float* lr_dev;
  const float* gscale;
  double lr, wd, log_b1, log_b2;
  float b1, omb1, b2, omb2, eps;
  uint32_t seed;
};

SBN_DEVFN uint32_t aw_mix(uint32_t x) {
  x = (x ^ (x >> 16)) * kAwHashA;
  x = (x ^ (x >> 15)) * kAwHashB;
  return x ^ (x >> 16);
}

// 1 / x within two steps of fp32, x >= FLT_MIN (only the parameters see it, not the states).
SBN_DEVFN float aw_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e as a float, -126 <= e <= 127.
SBN_DEVFN float aw_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Exponent of a block's scale from the bits of its largest magnitude: the
// codes of the block then lie below 2^8 (e4m3 reaches 448).
SBN_DEVFN int aw_scale_exp(uint32_t top_bits) { return max((int)(top_bits >> 23) - 127, -100); }

// The e4m3 grid at y >= 0 (below 2^8): three mantissa bits, a fixed step of
// 2^-9 below 2^-6. Adding 2^-6 to such a y puts its steps where a normal
// number has them, in the top three bits of the mantissa.
constexpr uint32_t kAwGridMask = 0xFFF00000u;
SBN_DEVFN float aw_grid_base(float y) { return y < 0.015625f ? 0.015625f : 0.f; }

// y to the grid: up from the point at or below it with probability (distance)
// / step, that is iff u < distance / step with u = h16 / 2^16 and the distance
// the 20 mantissa bits below the grid. A carry out of them does the step: it
// happens iff bits + (2^20 - 1 - 16 h16) >= 2^20, that is bits > 16 h16. The
// base is added rounding up: bits beyond the sum's last, which u * step never
// has, then still count as "above".
SBN_DEVFN float aw_round(float y, uint32_t h16) {
  const float base = aw_grid_base(y);
  const uint32_t w = __float_as_uint(__fadd_ru(y, base));
  return __fsub_rn(__uint_as_float((w + ((h16 << 4) ^ 0xFFFFFu)) & kAwGridMask), base);
}

// The same with the probability that keeps the expected square: between lo
// and lo + ulp iff u ((lo + ulp)^2 - lo^2) < y^2 - lo^2. No y > 0 becomes 0.
SBN_DEVFN float aw_round_root(float y, uint32_t h16) {
  const float base = aw_grid_base(y);
  const uint32_t w = __float_as_uint(__fadd_rz(y, base)) & kAwGridMask;
  const float lo = __fsub_rn(__uint_as_float(w), base);
  const float ulp = __uint_as_float((w & 0x7F800000u) - (3u << 23));
  // 16 random bits as a float in [0, 1); conversions would run at an eighth of the rate
  const float u = __fsub_rn(__uint_as_float(0x3F800000u | (h16 << 7)), 1.f);
  const bool up = __fmul_rn(__fmul_rn(u, ulp), __fmaf_rn(2.f, lo, ulp)) < __fmul_rn(__fsub_rn(y, lo), __fadd_rn(y, lo));
  const float q = up ? __fadd_rn(lo, ulp) : lo;
  return y > 0.f ? fmaxf(q, 1.f / 512.f) : q;
}

SBN_DEVFN void aw_decode2(uint16_t c, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  asm("{\n.reg .f16 l, h;\nmov.b32 {l, h}, %2;\ncvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}\n" : "=f"(a), "=f"(b) : "r"(h));
}
SBN_DEVFN uint16_t aw_encode2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}

// Eight consecutive fp32 (32-byte aligned) in one access.
SBN_DEVFN void aw_ld8(const float* p, float (&r)[8]) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "l"(p));
}
SBN_DEVFN void aw_st8(float* p, const float (&r)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]),
               "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}
SBN_DEVFN void aw_ld8(const uint16_t* p, float (&r)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = __uint_as_float(w[i] << 16);
    r[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
SBN_DEVFN void aw_st8(uint16_t* p, const float (&r)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(r[2 * i])) |
           ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(r[2 * i + 1])) << 16);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
SBN_DEVFN float aw_ld1(const float* p) { return *p; }
SBN_DEVFN float aw_ld1(const uint16_t* p) { return bf16_bits_to_float(*p); }
SBN_DEVFN void aw_st1(float* p, float x) { *p = x; }
SBN_DEVFN void aw_st1(uint16_t* p, float x) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// Eight elements from index i on, `have` of them inside the tensor (0..8);
// the others read as zero and are not written.
template <typename T>
SBN_DEVFN void aw_load(const T* p, size_t i, int have, bool vec, float (&r)[8]) {
  if (vec && have == 8) {
    aw_ld8(p + i, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = j < have ? aw_ld1(p + i + j) : 0.f;
  }
}
template <typename T>
SBN_DEVFN void aw_store(T* p, size_t i, int have, bool vec, const float (&r)[8]) {
  if (vec && have == 8) {
    aw_st8(p + i, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < have) aw_st1(p + i + j, r[j]);
  }
}

SBN_DEVFN void aw_load_codes(const uint8_t* p, size_t i, int have, bool vec, float scale, float (&r)[8]) {
  uint2 c = make_uint2(0u, 0u);
  if (vec && have == 8) {
    c = *reinterpret_cast<const uint2*>(p + i);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < have) (j < 4 ? c.x : c.y) |= (uint32_t)p[i + j] << (8 * (j & 3));
  }
  aw_decode2((uint16_t)c.x, r[0], r[1]);
  aw_decode2((uint16_t)(c.x >> 16), r[2], r[3]);
  aw_decode2((uint16_t)c.y, r[4], r[5]);
  aw_decode2((uint16_t)(c.y >> 16), r[6], r[7]);
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = __fmul_rn(r[j], scale);
}

// max(a, |b|) that keeps a NaN.
SBN_DEVFN float aw_max_abs(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(b)));
  return y;
}

// Codes of eight elements of a warp's block and the block's scale (lane 0).
// ROOT: r = sqrt(v), with the high half of the random words; else m, the low.
template <bool ROOT>
SBN_DEVFN void aw_store_codes(uint8_t* p, float* scale, size_t i, int have, bool vec, const float (&r)[8],
                              const uint32_t (&h)[8]) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = aw_max_abs(top, r[j]);
  uint32_t top_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top)), lost = 0u;
  if (top_bits >= 0x7F800000u) {   // the same for every lane: an infinity or a NaN somewhere in the block
    top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (isfinite(r[j])) top = fmaxf(top, fabsf(r[j]));
      else lost |= 1u << j;
    }
    top_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  }
  const int e = aw_scale_exp(top_bits);
  const float up = aw_pow2(7 - e);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = __fmul_rn(fabsf(r[j]), up);
    q[j] = ROOT ? aw_round_root(y, h[j] >> 16) : copysignf(aw_round(y, h[j] & 0xFFFFu), r[j]);
  }
  if (lost) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lost >> j & 1u) q[j] = __uint_as_float(0x7FC00000u);
  }
  uint2 c;
  c.x = (uint32_t)aw_encode2(q[0], q[1]) | ((uint32_t)aw_encode2(q[2], q[3]) << 16);
  c.y = (uint32_t)aw_encode2(q[4], q[5]) | ((uint32_t)aw_encode2(q[6], q[7]) << 16);
  if (vec && have == 8) {
    *reinterpret_cast<uint2*>(p + i) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < have) p[i + j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
  if ((threadIdx.x & 31) == 0) *scale = aw_pow2(e - 7);
}

template <typename P, typename G, int BITS, int N>
__global__ void __launch_bounds__(kAwThreads)
adamw_kernel(const __grid_constant__ AwTable<N> tab, const AwHyper hp) {
  griddep_wait();
  const int t = hp.step[0] + 1;
  const double lr = hp.lr_dev ? (double)*hp.lr_dev : hp.lr;
  const float gs = hp.gscale ? *hp.gscale : 1.f;
  // 1 - b^t = -expm1(t log b): accurate for every t
  const float bc1 = -expm1f((float)((double)t * hp.log_b1)), bc2 = -expm1f((float)((double)t * hp.log_b2));
  const float a = (float)(lr / (double)bc1);
  const float c2 = __fdiv_rn(1.f, __fsqrt_rn(bc2));
  const float dec = (float)(1.0 - lr * hp.wd);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t total = tab.first[tab.count];

  for (uint32_t s = blockIdx.x; s < total; s += gridDim.x) {
    int lo = 0, hi = tab.count;   // first[lo] <= s < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tab.first[mid] <= s) lo = mid;
      else hi = mid;
    }
    const AwEntry& e = tab.e[lo];
    const uint32_t blk = (s - tab.first[lo]) * (kAwThreads / 32) + warp;
    const size_t i = (size_t)blk * kAwBlock + 8 * lane;
    if ((size_t)blk * kAwBlock >= e.numel) continue;
    const int have = i >= e.numel ? 0 : (int)min((size_t)8, (size_t)e.numel - i);
    const bool vec = e.vec != 0u;
    P* pp = reinterpret_cast<P*>(e.p);
    float p[8], g[8], m[8], v[8];
    aw_load(pp, i, have, vec, p);
    aw_load(reinterpret_cast<const G*>(e.g), i, have, vec, g);
    if (BITS == 32) {
      aw_load(reinterpret_cast<const float*>(e.m), i, have, vec, m);
      aw_load(reinterpret_cast<const float*>(e.v), i, have, vec, v);
    } else {
      aw_load_codes(reinterpret_cast<const uint8_t*>(e.m), i, have, vec, e.ms[blk], m);
      aw_load_codes(reinterpret_cast<const uint8_t*>(e.v), i, have, vec, e.vs[blk], v);
    }
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = __fmul_rn(g[j], gs);
      const float v0 = BITS == 32 ? v[j] : __fmul_rn(v[j], v[j]);
      m[j] = __fadd_rn(__fmul_rn(hp.b1, m[j]), __fmul_rn(hp.omb1, gj));
      v[j] = __fadd_rn(__fmul_rn(hp.b2, v0), __fmul_rn(hp.omb2, __fmul_rn(gj, gj)));
      r[j] = __fsqrt_rn(v[j]);
      const float u = __fmul_rn(m[j], aw_rcp(__fadd_rn(__fmul_rn(r[j], c2), hp.eps)));
      p[j] = __fsub_rn(__fmul_rn(p[j], dec), __fmul_rn(a, u));
    }
    aw_store(pp, i, have, vec, p);
    if (sizeof(P) == 4 && e.copy) aw_store(e.copy, i, have, vec, p);
    if (BITS == 32) {
      aw_store(reinterpret_cast<float*>(e.m), i, have, vec, m);
      aw_store(reinterpret_cast<float*>(e.v), i, have, vec, v);
    } else {
      const uint32_t key = aw_mix(hp.seed + (uint32_t)t * kAwHashA + (tab.id0 + (uint32_t)lo) * kAwHashB);
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = aw_mix(((uint32_t)i + (uint32_t)j) ^ key);
      if (have < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= have) m[j] = r[j] = 0.f;   // behind the tensor's end
      }
      aw_store_codes<false>(reinterpret_cast<uint8_t*>(e.m), e.ms + blk, i, have, vec, m, h);
      aw_store_codes<true>(reinterpret_cast<uint8_t*>(e.v), e.vs + blk, i, have, vec, r, h);
    }
  }
  griddep_launch_dependents();
  // the last CTA advances the step, after every CTA has read it
  if (tab.last) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(reinterpret_cast<unsigned*>(hp.step) + 1, 1u) == gridDim.x - 1u) {
        hp.step[1] = 0;
        hp.step[0] = t;
      }
    }
  }
}

}  // namespace sbn
