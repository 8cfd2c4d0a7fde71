// Addressing and element helpers of the page-cache kernels (16-bit and MXFP4 records).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "tq_internal.h"

namespace tq {

// a / b for a >= 0, 0 < b < 2^31: in 32 bits where they suffice (a 64-bit division is about
// five times the instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// a * b for 0 <= a < 2^32: half the instructions of a full 64-bit product.
__device__ __forceinline__ int64_t times(uint32_t a, int64_t b) { return (int64_t)((uint64_t)a * (uint64_t)b); }

// Byte offset of cache row `slot`'s record for KV head 0 (or the page's own head); `soff` its
// scale bytes'. Pages and tokens fit 31 and 20 bits.
template <bool MX>
__device__ __forceinline__ int64_t record_offset(const PageView& p, int64_t slot, int64_t& soff) {
  const uint32_t pg = (uint32_t)(p.page_shift >= 0 ? slot >> p.page_shift : quotient(slot, p.page_size));
  const uint32_t t = (uint32_t)slot - pg * (uint32_t)p.page_size;
  if constexpr (MX) soff = times(pg, p.spage_b) + times(t, p.stok_b);
  return times(pg, p.page_b) + times(t, p.tok_b);
}

template <typename T>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t pack_rz(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <>
struct Half2<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t pack_rz(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// Two fp32 values to two e2m1 codes (low nibble first): to nearest, ties to the even code,
// magnitudes above 6 become 6.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b8 c; cvt.rn.satfinite.e2m1x2.f32 c, %2, %1; cvt.u32.u8 %0, c; }" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// The eight e2m1 codes of `w` as f16 pairs (exact): out[j] = codes 2j, 2j + 1.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&out)[4]) {
  asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}

// E8M0 scale byte as fp32: 2^(s - 127), NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fffffffu : s << 23);
}

// The same as bf16 bits.
__device__ __forceinline__ uint32_t e8m0_bf16(uint32_t s) { return s == 0 ? 0x0040u : s == 255 ? 0x7fffu : s << 7; }

}  // namespace tq
