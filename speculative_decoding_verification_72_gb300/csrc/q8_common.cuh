// The 8-bit paged cache and the pieces its kernels share.
//
// K and V are e4m3 codes [pages, Hkv, P, D] with one fp32 scale per page and
// head ([pages, Hkv]); a code stands for code * scale. A page's head is one
// contiguous tile of P * D bytes, so a run of tokens is read with full-width
// loads whatever the number of heads. Position p of request b is slot p % P of
// page table[b, p / P]; P is a power of two from 16 to 128.
#pragma once

#include <cuda_fp16.h>

#include "sv_common.cuh"

namespace sv {

struct Q8View {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* table;   // [B, max_pages]
  int32_t num_pages, Hkv, page_shift, max_pages;
};

// Page id of logical page lp of request b, or -1 if there is none.
__device__ __forceinline__ int q8_page(const Q8View& c, int b, int lp) {
  if (lp < 0 || lp >= c.max_pages) return -1;
  const int p = c.table[static_cast<int64_t>(b) * c.max_pages + lp];
  return p >= 0 && p < c.num_pages ? p : -1;
}

// Two e4m3 codes (the low 16 bits of w) as f16x2; exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ float2 half2_bits(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// Four floats as e4m3 codes, nearest-even; past the largest value (infinities
// too) saturates, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Codes times a factor, rounded to codes again (a change of scale). For a
// power of two the product is exact, so the only rounding is the last one.
__device__ __forceinline__ uint32_t e4m3_rescale4(uint32_t w, float f) {
  const float2 lo = half2_bits(e4m3x2_lo(w)), hi = half2_bits(e4m3x2_hi(w));
  return e4m3_pack4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of the smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8
// is e4m3's largest value), at least 2^-100 (an all-zero block) and at most
// 2^119 (so that 448 s is finite). Powers of two make every change of scale
// exact and cost e4m3, a floating type, no precision above its subnormals.
__device__ __forceinline__ int q8_need_exp(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 127;
  const int need = (bits & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7;
  return min(max(need, -100), 119);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Element types of q / new rows / outputs.
struct TypeF32 {
  static constexpr int kBytes = 4;
};
struct TypeBf16 {
  static constexpr int kBytes = 2;
  static constexpr int kExpBits = 8;
  static constexpr uint32_t kMma = 1;   // kind::f16's code of the type
  __device__ static float2 unpack2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
  __device__ static void unpack8(const uint4& w, float* f) { Elem<2>::unpack(w, f); }
  // max that hands on NaN
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static float value(uint16_t bits) { return __uint_as_float(static_cast<uint32_t>(bits) << 16); }
  __device__ static void load8(const void* p, float* f) { unpack8(*reinterpret_cast<const uint4*>(p), f); }
  __device__ static void load4(const void* p, float* f) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(w.x << 16);
    f[1] = __uint_as_float(w.x & 0xffff0000u);
    f[2] = __uint_as_float(w.y << 16);
    f[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  __device__ static uint32_t pack2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    return r;
  }
};
struct TypeF16 {
  static constexpr int kBytes = 2;
  static constexpr int kExpBits = 5;
  static constexpr uint32_t kMma = 0;
  __device__ static float2 unpack2(uint32_t w) { return half2_bits(w); }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static float value(uint16_t bits) { return __half2float(__ushort_as_half(bits)); }
  __device__ static void load8(const void* p, float* f) { unpack8(*reinterpret_cast<const uint4*>(p), f); }
  __device__ static void unpack8(const uint4& w, float* f) {
    const float2 a = half2_bits(w.x), b = half2_bits(w.y), c = half2_bits(w.z), d = half2_bits(w.w);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
  }
  __device__ static void load4(const void* p, float* f) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = half2_bits(w.x), b = half2_bits(w.y);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  }
  __device__ static uint32_t pack2(float a, float b) { return pack_half2(a, b); }
};

}  // namespace sv
