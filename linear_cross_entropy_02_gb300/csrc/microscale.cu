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
// Both kernels move memory and little else: a warp takes 256 consecutive
// elements of a row, eight per lane, so that reads and writes are whole lines;
// the four lanes of a block share its magnitude by two shuffles, and the four
// scale bytes that lie together in a scale tile leave as one word.
#include "head_device.cuh"
#include "head_internal.h"

namespace flce {

namespace {

constexpr int kChunk = 256;  // elements of a row per warp step

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

// Work of a warp: `seg` chunks of a row, part `part` of `parts`. Warp w of the
// grid takes tasks w, w + warps, ... in the order of (row, part).
struct Split {
  int64_t rows;  // rows to visit
  int parts, seg, chunks;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantParams p, const Split sp) {
  const int lane = threadIdx.x & 31;
  if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  const int64_t tasks = sp.rows * sp.parts;
  const int64_t k_tiles = (p.cols + kMxTileCols - 1) / kMxTileCols;
  const T* x = static_cast<const T*>(p.x);
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); task < tasks; task += warps) {
    const int64_t row = task / sp.parts;
    const int part = static_cast<int>(task - row * sp.parts);
    const int c0 = part * sp.seg, c1 = min(c0 + sp.seg, sp.chunks);
    const bool real = row < p.rows;  // rows that only fill the last scale tile are not read
#pragma unroll 2
    for (int ch = c0; ch < c1; ++ch) {
      const int64_t col = static_cast<int64_t>(ch) * kChunk + lane * 8;
      const bool in = real && col < p.cols;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
      if (in) {
        const T* q = x + row * p.ld_x + col;
        if constexpr (!VEC) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = to_float<T>(q[j]);
        } else if constexpr (sizeof(T) == 2) {
          const Raw<T, 8> r = load_raw<T, 8>(q);
          unpack<T, 8>(r, v);
        } else {
          const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
          v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
          v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
      }
      uint32_t top = 0;  // magnitudes as bit patterns: NaN is above infinity, both above every number
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t E = top >> 23;
      const uint32_t byte = E == 255u ? 255u : E > 2u ? E - 2u : 0u;
      if (in) {
        const float inv = E == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inv;
        const uint32_t c = E == 255u ? 0u : encode8(v);
        *reinterpret_cast<uint32_t*>(p.codes + row * (p.cols / 2) + col / 2) = c;
      }
      // the four blocks of a K-tile: lanes 0, 4, 8, 12 (and 16, ...)
      uint32_t word = in ? byte : 127u;
      word = word | (__shfl_down_sync(0xffffffffu, word, 4) << 8);
      word = (word & 0xFFFFu) | (__shfl_down_sync(0xffffffffu, word, 8) << 16);
      const int64_t kt = col / kMxTileCols;
      if ((lane & 15) == 0 && kt < k_tiles)
        *reinterpret_cast<uint32_t*>(p.scales + scale_word(row, kt, k_tiles)) = word;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t cols,
                                                            T* out, const Split sp) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  const int64_t tasks = sp.rows * sp.parts;
  const int64_t k_tiles = (cols + kMxTileCols - 1) / kMxTileCols;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); task < tasks; task += warps) {
    const int64_t row = task / sp.parts;
    const int part = static_cast<int>(task - row * sp.parts);
    const int c0 = part * sp.seg, c1 = min(c0 + sp.seg, sp.chunks);
#pragma unroll 2
    for (int ch = c0; ch < c1; ++ch) {
      const int64_t col = static_cast<int64_t>(ch) * kChunk + lane * 8;
      if (col >= cols) continue;
      const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes + row * (cols / 2) + col / 2));
      const float s = scale_value(__ldg(scales + scale_word(row, col / kMxTileCols, k_tiles) + (lane >> 2 & 3)));
      float v[8];
      decode8(c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
      T* o = out + row * cols + col;
      if constexpr (sizeof(T) == 2) {
        store_raw<T, 8>(o, pack<T, 8>(v));
      } else {
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
}

// Rows are cut into parts until every SM has its 64 warps, and no further: a
// part of several chunks keeps two loads per lane in flight.
Split split_rows(int64_t rows, int64_t cols, int sms) {
  Split s;
  s.rows = rows;
  s.chunks = static_cast<int>((cols + kChunk - 1) / kChunk);
  const int64_t want = 64LL * sms;
  int64_t parts = (want + rows - 1) / rows;
  if (parts > s.chunks) parts = s.chunks;
  s.seg = static_cast<int>((s.chunks + parts - 1) / parts);
  s.parts = (s.chunks + s.seg - 1) / s.seg;
  return s;
}

inline unsigned grid_of(const Split& s, int sms) {
  const int64_t want = (s.rows * s.parts + 7) / 8, most = 16LL * sms;
  return static_cast<unsigned>(want < most ? want : most);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantParams& p, int sms, cudaStream_t s) {
  const int64_t rows = (p.rows + kMxTileRows - 1) / kMxTileRows * kMxTileRows;
  const Split sp = split_rows(rows, p.cols, sms);
  const unsigned grid = grid_of(sp, sms);
  const int64_t es = p.dtype == FLCE_DTYPE_F32 ? 4 : 2;
  const bool vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ld_x * es % 16 == 0;
  if (p.dtype == FLCE_DTYPE_F32) {
    if (vec)
      mx_quantize_kernel<float, true><<<grid, 256, 0, s>>>(p, sp);
    else
      mx_quantize_kernel<float, false><<<grid, 256, 0, s>>>(p, sp);
  } else {
    if (vec)
      mx_quantize_kernel<uint16_t, true><<<grid, 256, 0, s>>>(p, sp);
    else
      mx_quantize_kernel<uint16_t, false><<<grid, 256, 0, s>>>(p, sp);
  }
  return cudaGetLastError();
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                 int out_dtype, int sms, cudaStream_t s) {
  const Split sp = split_rows(rows, cols, sms);
  const unsigned grid = grid_of(sp, sms);
  if (out_dtype == FLCE_DTYPE_F32)
    mx_dequantize_kernel<float><<<grid, 256, 0, s>>>(codes, scales, cols, static_cast<float*>(out), sp);
  else
    mx_dequantize_kernel<uint16_t><<<grid, 256, 0, s>>>(codes, scales, cols, static_cast<uint16_t*>(out), sp);
  return cudaGetLastError();
}

}  // namespace flce
