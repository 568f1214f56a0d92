// Microscaled formats (OCP Microscaling Formats v1.0): blocks of 32 values
// share one power-of-two scale, an E8M0 byte s standing for 2^(s - 127).
// The shared exponent is floor(log2(largest magnitude)) less the element
// type's largest exponent (2 for E2M1, 8 for E4M3), at least -127; elements
// are rounded to nearest even and saturate.  A block of zeros has scale byte
// 0.  A block that holds a NaN or an infinity, which E2M1 cannot express,
// gets the NaN scale 255 and reads back as NaN.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace moonep {

constexpr int kMxBlock = 32;

// Scale byte of a block whose largest magnitude has the bits `amax` (sign
// cleared; NaN and infinity compare above every finite value).
template <int EMAX>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = (int)(amax >> 23) - EMAX;  // biased exponent; 0 below the normals
  return (uint32_t)(b > 0 ? b : 0);
}

// The factor 2^(127 - s) that takes a value to its block's grid (exact for
// every finite block: s is at most 252), 0 for the NaN scale.
__device__ __forceinline__ float mx_inverse(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// The scale itself, 2^(s - 127); s = 0 is a subnormal, 255 NaN.
__device__ __forceinline__ float mx_value(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7fffffffu)
                   : (s ? __uint_as_float(s << 23) : __uint_as_float(0x00400000u));
}

// A pair of half-precision values as fp32.
__device__ __forceinline__ void mx_half2(uint32_t h, float *lo, float *hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(*lo), "=f"(*hi)
      : "r"(h));
}

// Eight values as packed E2M1 codes, value 0 in the lowest four bits.
__device__ __forceinline__ uint32_t mx_pack_e2m1(const float v[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight packed E2M1 codes as fp32, through half precision.
__device__ __forceinline__ void mx_e2m1x8(uint32_t w, float f[8]) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; i++) mx_half2(h[i], &f[2 * i], &f[2 * i + 1]);
}

// Four values as E4M3 codes, value 0 in the lowest byte.
__device__ __forceinline__ uint32_t mx_pack_e4m3(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n"
      " cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
      " mov.b32 %0, {a, b};\n}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return r;
}

// Two E4M3 codes (low 16 bits) as fp32, through half precision, which holds
// every E4M3 value.
__device__ __forceinline__ float2 mx_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("{\n .reg .b16 a;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}" : "=r"(h) : "r"(c));
  float2 f;
  mx_half2(h, &f.x, &f.y);
  return f;
}

// Eight bf16 values of a 16-byte vector as fp32.
__device__ __forceinline__ void bf16x8(uint4 v, float f[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 to_bf16x8(const float f[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude (as bits) of eight values, then of the four lanes that
// hold a block together.
__device__ __forceinline__ uint32_t mx_amax(const float f[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Rows of rank j's window that belong to a segment: the last entry of
// cu_seqlens[j], kept within the window.
__device__ __forceinline__ int used_rows(const int32_t *cu, int j, int EB, int NvS) {
  const int v = cu[(int64_t)j * EB + EB - 1];
  return v < 0 ? 0 : (v > NvS ? NvS : v);
}

}  // namespace moonep
