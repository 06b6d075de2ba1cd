// Device-side helpers shared by the operators around the head: element groups
// in bf16 and fp32, warp sums, asynchronous copies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace flce {

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<uint16_t>(uint16_t v) {  // bf16 bits
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
template <>
__device__ __forceinline__ float to_float<float>(float v) {
  return v;
}

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ uint16_t from_float<uint16_t>(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}

// E consecutive elements as they lie in memory: 16 bytes, or one element.
template <typename T, int E>
struct Raw {
  uint4 u;
};
template <typename T>
struct Raw<T, 1> {
  T u;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <typename T, int E>
__device__ __forceinline__ void unpack(const Raw<T, E>& r, float (&v)[E]) {
  if constexpr (E == 1) {
    v[0] = to_float<T>(r.u);
  } else {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
}

template <typename T, int E>
__device__ __forceinline__ Raw<T, E> pack(const float (&v)[E]) {
  Raw<T, E> r;
  if constexpr (E == 1) {
    r.u = from_float<T>(v[0]);
  } else if constexpr (sizeof(T) == 2) {
    r.u = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    r.u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  return r;
}

template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, E>*>(p);
}
template <typename T, int E>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, E>& r) {
  *reinterpret_cast<Raw<T, E>*>(p) = r;
}

// E consecutive weights (fp32 or bf16) from element i on.
template <int E>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int i, float (&v)[E]) {
  if (f32) {
    const float* p = static_cast<const float*>(w) + i;
    if constexpr (E == 1) {
      v[0] = __ldg(p);
    } else {
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p + j));
        v[j] = a.x;
        v[j + 1] = a.y;
        v[j + 2] = a.z;
        v[j + 3] = a.w;
      }
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(w) + i;
    if constexpr (E == 1) {
      v[0] = to_float<uint16_t>(__ldg(p));
    } else {
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(p + j));
        v[j] = __uint_as_float(a.x << 16);
        v[j + 1] = __uint_as_float(a.x & 0xFFFF0000u);
        v[j + 2] = __uint_as_float(a.y << 16);
        v[j + 3] = __uint_as_float(a.y & 0xFFFF0000u);
      }
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Asynchronous copy of BYTES (4 or 16) from global to shared memory, private to
// the issuing thread: it reads the bytes back itself after copies_wait.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* gmem) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(gmem), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace flce
