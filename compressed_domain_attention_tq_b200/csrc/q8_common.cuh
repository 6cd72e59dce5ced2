// q8_common.cuh -- what the kernels of the 8-bit block-scaled cache share: the
// two code formats, their exact conversion to f16, and row arithmetic.
//
// A cache row of a kv head is d codes of 8 bits; the rows of a block of
// `block` tokens share one fp32 scale, and a value is scale * code.  Codes are
// int8 in [-127, 127] or e4m3 in [-448, 448]; every one of them is exact in
// f16 (11 significand bits, exponents 2^-24 .. 2^15), so the tensor cores
// multiply the codes themselves and the scale is applied to the fp32 sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "tc_ptx.cuh"

namespace tq {
namespace q8 {

constexpr float kLog2e = 1.4426950408889634f;

// two fp32 operations of one instruction, each rounded to nearest
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "sub.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

struct Int8 {
  static constexpr float kMax = 127.0f;
  static constexpr bool kSignedZero = false;
  // byte place of a 32-bit word that cvt_word puts into half k of pair p
  static __host__ __device__ constexpr int place(int p, int k) { return p + 2 * k; }

  // c + 128 as the low byte of the f16 1024 + (c + 128), less 1152: exact
  static __device__ __forceinline__ uint32_t from_even_bytes(uint32_t w) {
    return tc::hsub2(tc::and_xor(w, 0x00ff00ffu, 0x64806480u), 0x64806480u);
  }
  static __device__ __forceinline__ void cvt_word(uint32_t w, uint32_t& p0, uint32_t& p1) {
    p0 = from_even_bytes(w);
    p1 = from_even_bytes(w >> 8);
  }
  // bytes x of two words a, b (x = 0..3) as the f16 pairs (a.x, b.x)
  static __device__ __forceinline__ void cvt_two(uint32_t a, uint32_t b, uint32_t (&p)[4]) {
    const uint32_t lo = tc::prmt(a, b, 0x5410), hi = tc::prmt(a, b, 0x7632);
    p[0] = from_even_bytes(lo);
    p[1] = from_even_bytes(lo >> 8);
    p[2] = from_even_bytes(hi);
    p[3] = from_even_bytes(hi >> 8);
  }
  static __device__ __forceinline__ float value(uint32_t w, int byte) {
    return (float)(int8_t)(w >> (8 * byte));
  }
  // y (already divided by the scale, finite or not) -> code: NaN 0, ends saturate
  static __device__ __forceinline__ uint32_t code(float y) {
    y = y != y ? 0.0f : fminf(fmaxf(y, -kMax), kMax);
    return (uint32_t)__float2int_rn(y) & 0xffu;
  }
  // four finite y with |y| <= kMax + 1/2: halves to even by the fp32 adder
  static __device__ __forceinline__ uint32_t codes4(float2 a, float2 b) {
    const float2 magic = make_float2(12582912.0f, 12582912.0f);  // 1.5 * 2^23
    a = add2(a, magic);
    b = add2(b, magic);
    return tc::prmt(tc::prmt(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                    tc::prmt(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  }
};

struct E4m3 {
  static constexpr float kMax = 448.0f;
  static constexpr bool kSignedZero = true;
  static __host__ __device__ constexpr int place(int p, int k) { return 2 * p + k; }

  static __device__ __forceinline__ uint32_t cvt2(uint32_t two) {
    uint32_t d;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(two));
    return d;
  }
  static __device__ __forceinline__ void cvt_word(uint32_t w, uint32_t& p0, uint32_t& p1) {
    p0 = cvt2(w);
    p1 = cvt2(w >> 16);
  }
  static __device__ __forceinline__ void cvt_two(uint32_t a, uint32_t b, uint32_t (&p)[4]) {
    const uint32_t lo = tc::prmt(a, b, 0x5140), hi = tc::prmt(a, b, 0x7362);
    p[0] = cvt2(lo);
    p[1] = cvt2(lo >> 16);
    p[2] = cvt2(hi);
    p[3] = cvt2(hi >> 16);
  }
  static __device__ __forceinline__ float value(uint32_t w, int byte) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(w >> (8 * byte)), __NV_E4M3);
    return __half2float(__half(h));
  }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(d)
        : "f"(lo), "f"(hi));
    return d;
  }
  static __device__ __forceinline__ uint32_t code(float y) {
    return pack2(y != y ? 0.0f : fminf(fmaxf(y, -kMax), kMax), 0.0f) & 0xffu;
  }
  static __device__ __forceinline__ uint32_t codes4(float2 a, float2 b) {
    return pack2(a.x, a.y) | (pack2(b.x, b.y) << 16);
  }
};

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The power of two by which a query row is multiplied: its largest element comes into
// [2^13, 2^14), as far as 2^e and 2^-e are normal numbers (every finite row stays below 2^16).
__device__ __forceinline__ int query_exponent(float top) {
  return top > 0.0f ? max(-114, min(126, 13 - ilogbf(top))) : 0;
}

// The exponent of a sum of weights (0 for sums of 0 and NaN).  States (m, l) and outputs are
// written divided by 2^this, with m raised by it: l is then in [1, 2), m within one of the
// logarithm of the sum, and an output no larger than twice the largest value.
__device__ __forceinline__ int sum_exponent(float l) {
  const int e = (int)(__float_as_uint(l) >> 23);
  return e == 0 || e >= 255 ? 0 : e - 127;
}

// Division by the block's scale s, correctly rounded: with r = RN(1/s), two
// residual steps q <- q + r (x - q s) end on RN(x / s) (Markstein's theorem:
// the last step starts from a faithful quotient and the residual of a fused
// multiply-add is exact).  That needs s and the residuals in the normal range,
// so scales outside [2^-90, 2^100] take the division instruction sequence;
// below that range a quotient under 2^-11 may be inexact, but its code is 0.
struct Divider {
  float s, r;
  bool fast;
  static __device__ __forceinline__ Divider by(float s) {
    return {s, __frcp_rn(s), s >= 0x1p-90f && s <= 0x1p100f};
  }
  __device__ __forceinline__ float2 quick(float2 x) const {  // (x - q s as fma(q, -s, x), which is exact too)
    const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s);
    float2 q = mul2(x, r2);
    q = fma2(fma2(q, s2, x), r2, q);
    return fma2(fma2(q, s2, x), r2, q);
  }
  __device__ __forceinline__ float any(float x) const { return s > 0.0f ? __fdiv_rn(x, s) : 0.0f; }
};

}  // namespace q8
}  // namespace tq
