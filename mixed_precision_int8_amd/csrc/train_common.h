// Eight values at a time of any type the training operators take, from and to
// memory that is aligned to its elements only (the hardware's vector accesses need
// no more than that; odd widths put every other row on an odd element).
#pragma once

#include "device_util.h"
#include "train_internal.h"

namespace llmint8 {

typedef float v8f __attribute__((ext_vector_type(8)));

template <int TYPE>
struct Elem {
  static constexpr int kBytes = TYPE == kF32 ? 4 : 2;
  struct __attribute__((packed, aligned(2))) P16 {
    uint32_t v[4];
  };
  struct __attribute__((packed, aligned(4))) P32 {
    float v[8];
  };
  using Raw = std::conditional_t<TYPE == kF32, P32, P16>;  // eight values as they lie in memory

  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    if constexpr (TYPE == kF32) return static_cast<const float*>(p)[i];
    else return Act16<TYPE == kBF16>::to_f32(static_cast<const uint16_t*>(p)[i]);
  }
  static __device__ __forceinline__ void put(void* p, int64_t i, float v) {
    if constexpr (TYPE == kF32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = Act16<TYPE == kBF16>::from_f32(v);
  }
  // values i .. i + 7, of which those below `end` exist (the others are 0)
  static __device__ __forceinline__ Raw load(const void* p, int64_t i, int64_t end) {
    Raw r;
    if (i + 8 <= end) {
      r = *reinterpret_cast<const Raw*>(static_cast<const char*>(p) + i * kBytes);
    } else if constexpr (TYPE == kF32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r.v[j] = i + j < end ? static_cast<const float*>(p)[i + j] : 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + i + 2 * j;
        r.v[j] = (i + 2 * j < end ? q[0] : 0u) | (i + 2 * j + 1 < end ? (uint32_t)q[1] << 16 : 0u);
      }
    }
    return r;
  }
  static __device__ __forceinline__ v8f wide(const Raw& r) {
    v8f f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (TYPE == kF32) f[j] = r.v[j];
      else f[j] = Act16<TYPE == kBF16>::to_f32(r.v[j >> 1] >> (16 * (j & 1)) & 0xffffu);
    }
    return f;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int64_t end, const v8f& f) {
    if (i + 8 <= end) {
      Raw r;
      if constexpr (TYPE == kF32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = f[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.v[j] = Act16<TYPE == kBF16>::pack2(f[2 * j], f[2 * j + 1]);
      }
      *reinterpret_cast<Raw*>(static_cast<char*>(p) + i * kBytes) = r;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < end) put(p, i + j, f[j]);
    }
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace llmint8
