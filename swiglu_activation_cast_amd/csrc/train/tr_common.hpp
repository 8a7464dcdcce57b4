// tr_common.hpp -- element types and small helpers of the training operators.
#pragma once
#include "../mx_kernels.hpp"

namespace mxt {

using mx::u32;
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float((u32)v << 16); }  // bf16 bits
__device__ __forceinline__ float to_f32(float v) { return v; }

// Rounded to nearest even (bf16 bits), or unchanged.
template <class T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 2) return (uint16_t)mx::pack_bf16(v, 0.0f);
  else return v;
}

}  // namespace mxt
