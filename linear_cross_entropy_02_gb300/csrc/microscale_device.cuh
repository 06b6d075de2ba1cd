// Device-side encoding of microscaled 4-bit numbers, shared by the quantisation
// kernels and the product that encodes a few tokens itself.
#pragma once

#include "head_device.cuh"
#include "head_internal.h"

namespace flce {

constexpr int kUnit = 16;  // elements that a lane encodes at a time: half a block

// Eight floats to eight codes: v[0] in the lowest four bits.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight codes to eight floats (every E2M1 value is exact in half precision).
__device__ __forceinline__ void decode8(uint32_t c, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h[i]));
  }
}

// 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : byte == 0u ? __uint_as_float(0x00400000u)
                                                                  : __uint_as_float(byte << 23);
}

// Byte offset of the word with the scales of row r, K-tile kt.
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t kt, int64_t k_tiles) {
  return ((r / kMxTileRows) * k_tiles + kt) * kMxTileBytes + (r % 32) * 16 + (r % kMxTileRows / 32) * 4;
}

// 16 elements from 16- or 32-byte aligned memory (wide), or one by one.
template <typename T>
__device__ __forceinline__ void load16(const T* p, bool wide, uint32_t (&r)[4 * sizeof(T)]) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r[8 * i]), "=r"(r[8 * i + 1]), "=r"(r[8 * i + 2]), "=r"(r[8 * i + 3]), "=r"(r[8 * i + 4]),
                     "=r"(r[8 * i + 5]), "=r"(r[8 * i + 6]), "=r"(r[8 * i + 7])
                   : "l"(p + i * 32 / sizeof(T)));
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = p[2 * i] | static_cast<uint32_t>(p[2 * i + 1]) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(p[i]);
  }
}
template <int N>
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[N], int i) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]),
               "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
               : "memory");
}

// The largest magnitude's biased exponent. Magnitudes are compared as bit
// patterns: NaN is above infinity, both above every number.
__device__ __forceinline__ uint32_t exponent16(const uint32_t (&r)[8]) {  // bf16 pairs
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, r[i] & 0x7FFF7FFFu);
  return max(m >> 16, m & 0xFFFFu) >> 7;
}
__device__ __forceinline__ uint32_t exponent16(const uint32_t (&r)[16]) {  // fp32
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, r[i] & 0x7FFFFFFFu);
  return m >> 23;
}

// The scale's byte for a block whose largest magnitude has biased exponent E.
__device__ __forceinline__ uint32_t scale_byte(uint32_t E) { return E == 255u ? 255u : E > 2u ? E - 2u : 0u; }

// The 16 codes of a unit (loaded by load16) in a block with that exponent.
template <int N>
__device__ __forceinline__ uint2 encode16(const uint32_t (&raw)[N], uint32_t E) {
  const float inv = E == 255u ? 0.f : __uint_as_float((254u - scale_byte(E)) << 23);
  uint2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (N == 8) {
        const uint32_t w = raw[h * 4 + j / 2];
        v[j] = __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16) * inv;
      } else {
        v[j] = __uint_as_float(raw[h * 8 + j]) * inv;
      }
    }
    (h ? c.y : c.x) = E == 255u ? 0u : encode8(v);
  }
  return c;
}

}  // namespace flce
