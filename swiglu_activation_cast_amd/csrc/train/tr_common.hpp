// tr_common.hpp -- element types and small helpers of the training operators.
#pragma once
#include "../mx_device.hpp"

namespace mxt {

using mx::u32;
typedef u32 u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Names the global address space: kernel parameters are generic pointers in a
// struct, through which the compiler would emit flat accesses.
template <class T>
__device__ __forceinline__ __attribute__((address_space(1))) T *gptr(T *p) {
  return (__attribute__((address_space(1))) T *)p;
}

// p + off bytes, with p wave-uniform and off per lane (scalar base, 32-bit
// offset).
template <class T>
__device__ __forceinline__ T *byte_off(T *p, u32 off) {
  return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(p) + off);
}

// Workgroups are dealt to the eight XCDs in turn: the work item of workgroup b
// of n that gives each XCD one contiguous range of items (the last n % 8 stay).
__device__ __forceinline__ u32 xcd_remap(u32 b, u32 n) {
  const u32 full = n - n % 8u;
  return b >= full ? b : (b % 8u) * (full / 8u) + b / 8u;
}

__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float((u32)v << 16); }  // bf16 bits
__device__ __forceinline__ float to_f32(float v) { return v; }

// Rounded to nearest even (bf16 bits), or unchanged.
template <class T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 2) return (uint16_t)mx::pack_bf16(v, 0.0f);
  else return v;
}

}  // namespace mxt
