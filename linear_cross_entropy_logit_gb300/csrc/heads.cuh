// Values of heads between memory and registers, packed in twos for the fp32 pipe.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace flce {

// N consecutive values as they lie in memory.
template <typename T, int N>
struct Raw {
  static constexpr int kWords = N * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // Values 2 i and 2 i + 1, packed.
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (sizeof(T) == 4)
      return pack_u32x2(w[2 * i], w[2 * i + 1]);
    else
      return pack_u32x2(w[i] << 16, w[i] & 0xffff0000u);
  }
};
// N values, packed in twos.
template <typename T, int N>
__device__ __forceinline__ void store_values(T* p, const uint64_t* x) {
  constexpr int kWords = N * sizeof(T) / 4;
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float a, b;
    unpack_f32x2(x[i], a, b);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(a);
      w[2 * i + 1] = __float_as_uint(b);
    } else {
      w[i] = pack_bf16x2(a, b);
    }
  }
  if constexpr (kWords == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

}  // namespace flce
