// Device-side encoding of 8-bit checkpoints: E4M3 codes with one power of two (E8M0)
// for each 32 consecutive elements of a row, the least that keeps the largest
// magnitude within 448, so that nothing saturates. An element's error is at most half
// a step of its four significant bits (2^-4 of it), or 2^-10 of the block's power of
// two where that is more (below 2^-14 of the largest magnitude at most). Whatever the
// power of two, an element above 2^-6 of it is rounded alike: it is a floating-point grid.
#pragma once

#include "head_device.cuh"
#include "microscale_device.cuh"

namespace flce {

constexpr int kCheckpointBlock = 32;
// The largest scale's byte, 2^120: of blocks with a magnitude above 1.75 2^127. There the code above 240 would stand
// for 2^128, which fp32 does not hold, so that 240 is the largest (1.9375 2^127 and more are still within 2^-4).
constexpr uint32_t kTopScale = 247;

__host__ __device__ __forceinline__ int64_t checkpoint_blocks(int64_t hidden) {
  return (hidden + kCheckpointBlock - 1) / kCheckpointBlock;
}

// The scale's byte (exponent + 127) for a block whose largest magnitude has these
// bits: 448 = 1.75 2^8, so the exponent is 8 less than the magnitude's, 7 less if its
// significand is above 1.75. Infinity and NaN give the NaN scale, 255.
__device__ __forceinline__ uint32_t checkpoint_scale(uint32_t bits) {
  const int exponent = static_cast<int>(bits >> 23);
  if (exponent == 255) return 255u;
  const int byte = exponent - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(byte > 0 ? byte : 0);
}

// Two floats to two codes, lo in the lower byte.
__device__ __forceinline__ uint32_t encode2_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// E codes, packed from the lowest byte on, times `scale`.
template <int E>
__device__ __forceinline__ void read_codes(const uint32_t (&words)[E == 8 ? 2 : 1], float scale, float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < (E + 1) / 2; ++i) {
    const uint16_t two = static_cast<uint16_t>(words[i / 2] >> (i % 2 * 16));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));  // exact
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
    v[2 * i] = lo * scale;
    if constexpr (E > 1) v[2 * i + 1] = hi * scale;
  }
}

// A vector of a checkpoint as it is held.
template <int E>
struct CodeVector {
  uint32_t words[E == 8 ? 2 : 1];
  float scale;
};
template <typename T, int E>
__device__ __forceinline__ void unpack(const CodeVector<E>& r, float (&v)[E]) {
  read_codes<E>(r.words, r.scale, v);
}
// One that need not lie on the blocks' boundaries: elements from `second` on have the next scale,
// and those outside of [from, to) are not the row's.
template <int E>
struct ShiftedCodes {
  uint32_t words[E == 8 ? 2 : 1];
  float scale, next;
  int second, from, to;
};
template <typename T, int E>
__device__ __forceinline__ void unpack(const ShiftedCodes<E>& r, float (&v)[E]) {
  read_codes<E>(r.words, 1.f, v);
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = e >= r.from && e < r.to ? v[e] * (e < r.second ? r.scale : r.next) : 0.f;
}

// Encodes vector `vec` of a row: codes [rows, hidden], scales [rows, blocks]. Called by
// whole warps, `vec` rising by one from lane to lane over groups of min(32 / E, lanes);
// lanes that are not `valid` have no part of the row.
template <typename T, int E>
__device__ __forceinline__ void keep_vector(const Raw<T, E>& raw, int64_t vec, bool valid, int lanes, uint8_t* codes,
                                            uint8_t* scales, int64_t row, int64_t hidden) {
  float v[E];
  uint32_t most = 0;
  if (valid) {
    unpack<T, E>(raw, v);
#pragma unroll
    for (int e = 0; e < E; ++e) most = max(most, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  }
  const int group = min(kCheckpointBlock / E, lanes);
  if (E == 1 && lanes == 32) {
    most = __reduce_max_sync(0xffffffffu, most);
  } else {
    for (int o = group >> 1; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if (!valid) return;
  const uint32_t byte = checkpoint_scale(most);
  // 2^-e; a block of NaN has codes of zero
  const float inv = byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] *= inv;
  if (byte == kTopScale) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fminf(fmaxf(v[e], -240.f), 240.f);
  }
  uint32_t words[E == 8 ? 2 : 1] = {};
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float hi = E > 1 ? v[E > 1 ? e + 1 : 0] : 0.f;
    words[e / 4] |= (byte == 255u ? 0u : encode2_e4m3(v[e], hi)) << (e % 4 * 8);
  }
  uint8_t* to = codes + row * hidden + vec * E;
  if constexpr (E == 8)
    *reinterpret_cast<uint2*>(to) = make_uint2(words[0], words[1]);
  else if constexpr (E == 4)
    *reinterpret_cast<uint32_t*>(to) = words[0];
  else
    *to = static_cast<uint8_t>(words[0]);
  if (vec * E % kCheckpointBlock == 0) scales[row * checkpoint_blocks(hidden) + vec * E / kCheckpointBlock] = static_cast<uint8_t>(byte);
}

}  // namespace flce
