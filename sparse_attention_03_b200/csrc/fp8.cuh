// Device helpers of the paged 8-bit caches: e4m3 codes, power-of-two scales and
// the geometry of a row.
#pragma once

#include "common.cuh"
#include "fp8.h"

namespace lsa {

// Two fp32 values -> two e4m3 codes (round to nearest even; the callers keep |x| <= 448).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp16 -> two e4m3 codes, and back (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t f16_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// hi = e4m3(x), lo = e4m3((x - hi) * k) of two fp16 values; k a power of two (the
// difference is exact in fp16: hi has the value's exponent and fewer bits).
template <int K>
__device__ __forceinline__ void split_e4m3(uint32_t h2, uint32_t& hi, uint32_t& lo) {
  constexpr uint32_t k2 = K == 16 ? 0x4c004c00u : 0x54005400u;  // fp16 16 and 64
  static_assert(K == 16 || K == 64, "the fp16 constants above");
  hi = e4m3x2_f16(h2);
  uint32_t d;
  asm("{\n .reg .b32 t;\n sub.rn.f16x2 t, %1, %2;\n mul.rn.f16x2 %0, t, %3;\n}\n" : "=r"(d) : "r"(h2), "r"(f16_e4m3x2(hi)), "r"(k2));
  lo = e4m3x2_f16(d);
}

// The scale's exponent for a vector whose largest magnitude has these bf16 bits
// (sign cleared): the smallest e with amax <= 448 * 2^e, 448 = 1.75 * 2^8, at
// least -126. A zero vector takes e = 0. The caller handles non-finite bits.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  const int e = (int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ bool bf16_finite(uint32_t abs_bits) { return abs_bits < 0x7f80u; }
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Two fp32 -> packed bf16, round to nearest even, NaN kept.
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The larger of the packed magnitudes (bf16 bits order like their magnitudes).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t acc, uint32_t v) { return __vmaxu2(acc, v & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t fold_max(uint32_t m) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
  return max(m & 0xffffu, m >> 16);
}

// Eight bf16 (16 bytes) -> eight codes, each element times inv (a power of two).
__device__ __forceinline__ uint2 quant8(uint4 v, float inv) {
  uint2 r;
  r.x = e4m3x2(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv) | e4m3x2(bf16_lo(v.y) * inv, bf16_hi(v.y) * inv) << 16;
  r.y = e4m3x2(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv) | e4m3x2(bf16_lo(v.w) * inv, bf16_hi(v.w) * inv) << 16;
  return r;
}

// Where a row's keys live and how many it sees: clamped, and flagged by the
// thread that reports. seq -1: a padding row (or an unknown sequence, then
// `pad` is false): no keys.
struct PagedGeom {
  int seq;
  bool pad;
  int64_t nvis;
};
__device__ __forceinline__ PagedGeom paged_geom(const PagedRows& a, int r, bool report) {
  PagedGeom g;
  g.pad = false;
  g.nvis = 0;
  g.seq = a.seq_of_row ? a.seq_of_row[r] : r;
  const int p = a.pos[r];  // asked for together with the sequence
  if (g.seq < 0 || g.seq >= a.n_seq) {
    g.pad = g.seq == -1;
    if (report && !g.pad) flag_error(a.err, LSA_DEVERR_SEQ);
    g.seq = -1;
    return g;
  }
  const int64_t room = min64(a.max_len, (int64_t)a.max_pages * kPage);
  g.nvis = (int64_t)p + 1;
  if (p < 0 || g.nvis > room) {
    if (report) flag_error(a.err, LSA_DEVERR_POS);
    g.nvis = max64(0, min64(g.nvis, room));
  }
  return g;
}
__device__ __forceinline__ bool page_ok(int page, int n_pages) { return (unsigned)page < (unsigned)n_pages; }

}  // namespace lsa
