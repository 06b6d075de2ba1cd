// Microscaled 4-bit matrices (OCP Microscaling Formats v1.0, MXFP4): encoding
// and decoding. E2M1 elements, one E8M0 scale per 32 elements of a row.
//
// The scale of a block is a power of two taken from the exponent bits of its
// largest magnitude: with a biased exponent E of that magnitude, the scale's
// byte is max(E - 2, 0) (2 is the exponent of 4, the largest power of two among
// the codes), and 255, the NaN scale, for E = 255 (an infinity or a NaN).
// x 2^-e is then exact, and the conversion instruction rounds it to the nearest
// code, ties to the even one, at most 6.
//
// Both kernels move memory and little else. A lane takes 16 consecutive elements,
// one 32-byte load of bf16, and the two lanes of a block share its magnitude by
// one shuffle. The matrix is taken as one sequence of such units, whatever its
// width, by CTAs that do a fixed number of them and leave. Four scale bytes that
// lie together in a scale tile leave as one word where all of a row's tiles are
// whole. 128256 x 4096 bf16: 220 us to write (6.0 TB/s), 193 to read back (6.9).
#include "head_internal.h"
#include "microscale_device.cuh"

namespace flce {

namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 2;      // units per thread, their loads in flight together

struct Shape {
  uint32_t units_per_row;
  int64_t units;      // of the whole matrix
  int64_t work_ctas;  // CTAs for them; the rest fill the scale tiles' other places
  int64_t k_tiles;
};

Shape shape_of(int64_t rows, int64_t cols) {
  Shape s;
  s.units_per_row = static_cast<uint32_t>(cols / kUnit);
  s.units = rows * s.units_per_row;
  s.work_ctas = (s.units + kThreads * kSteps - 1) / (kThreads * kSteps);
  s.k_tiles = (cols + kMxTileCols - 1) / kMxTileCols;
  return s;
}

// Row and unit within the row of a unit.
__device__ __forceinline__ void place_of(int64_t unit, uint32_t per_row, int64_t& row, uint32_t& u) {
  if (unit >> 32 == 0) {
    const uint32_t r = static_cast<uint32_t>(unit) / per_row;
    row = r;
    u = static_cast<uint32_t>(unit) - r * per_row;
  } else {
    row = unit / per_row;
    u = static_cast<uint32_t>(unit - row * per_row);
  }
}

// WORDS: cols is a multiple of 128, so that eight lanes hold a whole scale word.
template <typename T, bool WORDS>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const MxQuantParams p, const Shape sh, const bool wide) {
  if (blockIdx.x >= sh.work_ctas) {
    // places without a block hold 127: rows beyond the last, blocks beyond the width
    const int64_t all = (p.rows + kMxTileRows - 1) / kMxTileRows * kMxTileRows;
    const int blocks = static_cast<int>(p.cols / kMxBlock);
    const int64_t step = static_cast<int64_t>(gridDim.x - sh.work_ctas) * kThreads;
    const int64_t first = (blockIdx.x - sh.work_ctas) * kThreads + threadIdx.x;
    for (int64_t i = first; i < (all - p.rows) * sh.k_tiles; i += step)
      *reinterpret_cast<uint32_t*>(p.scales + scale_word(p.rows + i / sh.k_tiles, i % sh.k_tiles, sh.k_tiles)) = 0x7F7F7F7Fu;
    if (!WORDS)
      for (int64_t row = first; row < p.rows; row += step)
        for (int b = blocks; b < sh.k_tiles * 4; ++b) p.scales[scale_word(row, b / 4, sh.k_tiles) + b % 4] = 127;
    return;
  }
  const T* x = static_cast<const T*>(p.x);
  uint32_t raw[kSteps][4 * sizeof(T)];
  int64_t row[kSteps];
  uint32_t u[kSteps];
  bool in[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int64_t unit = (blockIdx.x * static_cast<int64_t>(kSteps) + k) * kThreads + threadIdx.x;
    in[k] = unit < sh.units;
    if (in[k]) {
      place_of(unit, sh.units_per_row, row[k], u[k]);
      load16<T>(x + row[k] * p.ld_x + static_cast<int64_t>(u[k]) * kUnit, wide, raw[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    uint32_t E = in[k] ? exponent16(raw[k]) : 0;
    E = max(E, __shfl_xor_sync(0xffffffffu, E, 1));
    const uint32_t byte = scale_byte(E);
    uint32_t word = byte;
    if (WORDS) {
      word |= __shfl_down_sync(0xffffffffu, word, 2) << 8;
      word = (word & 0xFFFFu) | __shfl_down_sync(0xffffffffu, word, 4) << 16;
    }
    if (!in[k]) continue;
    if (WORDS) {
      if ((threadIdx.x & 7) == 0)
        *reinterpret_cast<uint32_t*>(p.scales + scale_word(row[k], u[k] / 8, sh.k_tiles)) = word;
    } else if ((threadIdx.x & 1) == 0) {
      p.scales[scale_word(row[k], u[k] / 8, sh.k_tiles) + (u[k] / 2 & 3)] = static_cast<uint8_t>(byte);
    }
    *reinterpret_cast<uint2*>(p.codes + row[k] * (p.cols / 2) + u[k] * 8) = encode16(raw[k], E);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, T* out, const Shape sh) {
  uint2 c[kSteps];
  uint32_t byte[kSteps];
  int64_t unit[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    unit[k] = (blockIdx.x * static_cast<int64_t>(kSteps) + k) * kThreads + threadIdx.x;
    if (unit[k] < sh.units) {
      int64_t row;
      uint32_t u;
      place_of(unit[k], sh.units_per_row, row, u);
      c[k] = __ldg(reinterpret_cast<const uint2*>(codes) + unit[k]);
      byte[k] = __ldg(scales + scale_word(row, u / 8, sh.k_tiles) + (u / 2 & 3));
    }
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    if (unit[k] >= sh.units) continue;
    const float s = scale_value(byte[k]);
    uint32_t r[4 * sizeof(T)];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      decode8(h ? c[k].y : c[k].x, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] *= s;
        if constexpr (sizeof(T) == 4) r[h * 8 + j] = __float_as_uint(v[j]);
      }
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[h * 4 + j] = pack_bf16(v[2 * j], v[2 * j + 1]);
      }
    }
    T* o = out + unit[k] * kUnit;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) store32(o + i * 32 / sizeof(T), r, 8 * i);
  }
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantParams& p, int sms, cudaStream_t s) {
  const Shape sh = shape_of(p.rows, p.cols);
  const int64_t es = p.dtype == FLCE_DTYPE_F32 ? 4 : 2;
  const bool wide = reinterpret_cast<uintptr_t>(p.x) % 32 == 0 && p.ld_x * es % 32 == 0;
  const bool words = p.cols % kMxTileCols == 0;
  const int64_t pad = (words ? 0 : p.rows) + (kMxTileRows - p.rows % kMxTileRows) % kMxTileRows * sh.k_tiles;
  const int64_t pad_ctas = (pad + kThreads - 1) / kThreads;
  const int64_t grid = sh.work_ctas + (pad_ctas < sms ? pad_ctas : sms);
  if (grid >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(grid);
  if (p.dtype == FLCE_DTYPE_F32) {
    if (words)
      mx_quantize_kernel<float, true><<<g, kThreads, 0, s>>>(p, sh, wide);
    else
      mx_quantize_kernel<float, false><<<g, kThreads, 0, s>>>(p, sh, wide);
  } else {
    if (words)
      mx_quantize_kernel<uint16_t, true><<<g, kThreads, 0, s>>>(p, sh, wide);
    else
      mx_quantize_kernel<uint16_t, false><<<g, kThreads, 0, s>>>(p, sh, wide);
  }
  return cudaGetLastError();
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                 int out_dtype, cudaStream_t s) {
  const Shape sh = shape_of(rows, cols);
  if (sh.work_ctas >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(sh.work_ctas);
  if (out_dtype == FLCE_DTYPE_F32)
    mx_dequantize_kernel<float><<<g, kThreads, 0, s>>>(codes, scales, static_cast<float*>(out), sh);
  else
    mx_dequantize_kernel<uint16_t><<<g, kThreads, 0, s>>>(codes, scales, static_cast<uint16_t*>(out), sh);
  return cudaGetLastError();
}

}  // namespace flce
