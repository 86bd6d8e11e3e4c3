// q8_common.cuh -- the 8-bit key/value cache: where a position's codes and
// exponent lie, and the conversions between e4m3 codes, f16 and bf16.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace ddt {

// Device view of ddt_q8_cache.
struct Q8View {
  uint8_t *kc, *vc;
  int8_t *ke, *ve;
  const int32_t* page_table;  // null: dense
  int page_size, max_pages, num_pages;
  int page_log2;              // -1: page_size is no power of two
  int64_t t_max;
  int hkv, d;
  int block_log2;
  int64_t blocks_per;         // exponent rows per sequence (dense) or page (paged)
};

// Cache row (token) of position t and its exponent row, or row -1 when the
// position lies outside the cache.
struct Q8Place {
  int64_t row, blk;
};
__device__ __forceinline__ Q8Place q8_place(const Q8View& c, int b, int64_t t) {
  Q8Place p{-1, -1};
  if (t < 0) return p;
  if (c.page_table == nullptr) {
    if (t < c.t_max) {
      p.row = (int64_t)b * c.t_max + t;
      p.blk = (int64_t)b * c.blocks_per + (t >> c.block_log2);
    }
    return p;
  }
  if (t >= (int64_t)c.max_pages * c.page_size) return p;
  const int pi = c.page_log2 >= 0 ? (int)((uint32_t)t >> c.page_log2)
                                  : (int)((uint32_t)t / (uint32_t)c.page_size);
  const int slot = (int)((uint32_t)t - (uint32_t)pi * (uint32_t)c.page_size);
  const int pg = c.page_table[(int64_t)b * c.max_pages + pi];
  if ((uint32_t)pg < (uint32_t)c.num_pages) {
    p.row = (int64_t)pg * c.page_size + slot;
    p.blk = (int64_t)pg * c.blocks_per + (slot >> c.block_log2);
  }
  return p;
}

__device__ __forceinline__ int q8_exp(int e) { return min(max(e, DDT_Q8_EXP_MIN), DDT_Q8_EXP_MAX); }
// 2^e for |e| <= 126.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Two e4m3 codes (low byte first) -> two f16, exactly: e4m3 is a subset of f16,
// and its NaN code stays NaN.  (The same by integers, a byte permute, a shift
// and a mask for each pair, takes more issue slots than the conversion costs: at
// the step that took it, 575 us against 554 us for 8 trees of 257 rows over 8192
// tokens, 216 us against 211 us for 32 ragged decoding steps.)
__device__ __forceinline__ uint32_t codes_to_f16(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// Bytes 0, 1 (lo) or 2, 3 (hi) of w.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return codes_to_f16((uint16_t)w); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return codes_to_f16((uint16_t)(w >> 16)); }
// Byte I of a and of b.
template <int I>
__device__ __forceinline__ uint32_t codes_of(uint32_t a, uint32_t b) {
  return codes_to_f16((uint16_t)prmt(a, b, 0x0040 + 0x0011 * I));
}
// What a code counts for in a block with the stored exponent e.
__device__ __forceinline__ float q8_scale(int e) {
  return e == DDT_Q8_EXP_NAN ? __int_as_float(0x7FC00000) : pow2i(q8_exp(e));
}
// Two floats -> two e4m3 codes (lo in the low byte), nearest-even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The softmax's reference for a largest exponent `top`: top - head, or top itself
// where the difference does not come out within head + slack of it (|top| beyond
// 2^26, whose last place is 8 and more), so that 2^(top - reference) fits f16.
__device__ __forceinline__ float reference_below(float top, float head, float slack) {
  const float to = top - head;
  return top - to <= head + slack ? to : top;
}

// ld_stream_v4 where `there`, zeros (and no access) elsewhere.
__device__ __forceinline__ uint4 ld_stream_v4_if(const void* p, bool there) {
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"((uint32_t)there));
  return r;
}

// The larger magnitude's bits of two packed bf16.
__device__ __forceinline__ uint32_t max_bf16(uint32_t w) { return max(w & 0x7FFFu, (w >> 16) & 0x7FFFu); }
// Magnitude bits of packed bf16 pairs, half by half.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
// The larger magnitude bits of the finite ones among two packed bf16 and m.
__device__ __forceinline__ uint32_t max_finite_bf16(uint32_t m, uint32_t w) {
  const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  if (lo < 0x7F80u) m = max(m, lo);
  if (hi < 0x7F80u) m = max(m, hi);
  return m;
}


// Exponent e with amax (bf16 magnitude bits, finite) * 2^-e in [2^top, 2^(top+1)).
__device__ __forceinline__ int f16_exponent(uint32_t amax_bits, int top) {
  return amax_bits < 0x80u ? -126 - top : (int)(amax_bits >> 7) - 127 - top;
}
// Exponent of a tree row as f16: its amax in [2^8, 2^9), as large as codes.
__device__ __forceinline__ int tree_exponent(uint32_t amax_bits) {
  return q8_exp(f16_exponent(amax_bits, 8));
}
// Two packed bf16 -> two f16 scaled by `inv` (a power of two).
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float inv) {
  return f32x2_to_f16x2(bf16_lo(w) * inv, bf16_hi(w) * inv);
}

// Tree V values from 2^57 on, infinities and NaN are no operands of the
// products, where even a weight of 0 would make NaN of them: they count as 0
// there, and as infinities (or NaN) in the rows whose mask shows them.
constexpr uint32_t kWildBits = (127 + 57) << 7;  // magnitude bits of bf16 2^57
__device__ __forceinline__ bool is_wild(uint32_t bf16_bits) { return (bf16_bits & 0x7FFFu) >= kWildBits; }
__device__ __forceinline__ bool has_wild(uint32_t w) { return is_wild(w) || is_wild(w >> 16); }
// Two packed bf16, wild ones as 0.
__device__ __forceinline__ uint32_t tame_bf16x2(uint32_t w) {
  if (is_wild(w)) w &= 0xFFFF0000u;
  if (is_wild(w >> 16)) w &= 0x0000FFFFu;
  return w;
}
// What a wild value counts for where it is seen.
__device__ __forceinline__ float wild_value(uint32_t bf16_bits) {
  return (bf16_bits & 0x7FFFu) > 0x7F80u ? __int_as_float(0x7FC00000)
                                         : (bf16_bits & 0x8000u) ? -INFINITY : INFINITY;
}

}  // namespace ddt
