// Codes of the quantised cache and 16-bit values, to and from fp32. Every
// conversion is one rounding to nearest even, or exact. GPU-library only.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvc.h"

namespace kvc {

constexpr float kE4m3Peak = 448.f, kInt8Peak = 127.f, kE2m1Peak = 2688.f;  // largest |y|: 2688 = 6 * 448
constexpr float kRowFloor = 0x1p-96f;  // rows below it are stored as zero; 1 / s stays finite above

// ---- 16-bit values
__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ inline float2 half2_f32(uint32_t w) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(w));
  return r;
}
__device__ inline uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ inline uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <uint32_t DT>
__device__ inline float2 unpack16(uint32_t w) {
  if (DT == KVC_DTYPE_BF16) return make_float2(bf16_lo(w), bf16_hi(w));
  return half2_f32(w);
}
template <uint32_t DT>
__device__ inline uint32_t pack16(float lo, float hi) {
  return DT == KVC_DTYPE_BF16 ? pack_bf16(lo, hi) : pack_half(lo, hi);
}

// ---- fp32 -> codes (saturating, nearest even)
__device__ inline uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// eight at once, y[0] in the lowest bits
__device__ inline uint32_t e2m1x8(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}
// round to nearest even, clipped to 127: in the low byte of x + 1.5 * 2^23
__device__ inline uint32_t int8_bits(float x) {
  return __float_as_uint(fminf(fmaxf(x, -127.f), 127.f) + 12582912.f);
}

// ---- codes -> half pairs (exact)
__device__ inline uint32_t e4m3x2_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ inline uint32_t e2m1x2_half2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}
__device__ inline float e4m3_f32(uint32_t byte) { return half2_f32(e4m3x2_half2(byte)).x; }
// signed byte `i` of w as fp32: 2^23 + (b + 128) put together as bits, less 2^23 + 128
template <int I>
__device__ inline float int8_f32(uint32_t w) {
  return __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7440u + I)) - 8388736.f;
}

}  // namespace kvc
