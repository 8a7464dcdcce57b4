// tr_host.hpp -- what the entry points share on the host: checks and launches.
#pragma once
#include <hip/hip_runtime.h>
#include <algorithm>
#include <cmath>
#include <limits.h>
#include <stdint.h>

#include "mxtrain.h"

namespace mxt {

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Elements of a [rows, cols] matrix with row stride ld, counted from its
// base, fit int64 with room for the element size and a batch on top.
inline bool extent_ok(int64_t rows, int64_t cols, int64_t ld) {
  int64_t r;
  if (rows == 0 || cols == 0) return true;
  return !__builtin_mul_overflow(rows - 1, ld, &r) && !__builtin_add_overflow(r, cols, &r) && r < (INT64_MAX >> 4);
}

template <class Args>
mxtrain_status launch(const void *kernel, int64_t blocks, int threads, const Args &a, void *stream, unsigned lds = 0) {
  // grid x times block x stays below 2^31
  if (blocks <= 0 || blocks > (int64_t)INT32_MAX / threads) return MXTRAIN_ERR_OVERFLOW;
  Args copy = a;
  void *kargs[] = {&copy};
  const hipError_t err =
      hipLaunchKernel(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), kargs, lds, (hipStream_t)stream);
  return err == hipSuccess ? MXTRAIN_OK : MXTRAIN_ERR_LAUNCH;
}

// Compute units of the current device.  They decide tile sizes and how many rows
// a workgroup walks, and with them the order of sums: a result's last bits are
// those of devices with as many.
inline int cu_count() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1)
    return 256;
  return cus;
}

inline bool type_ok(int t) { return t == MXTRAIN_BF16 || t == MXTRAIN_F32; }
inline int size_of(int t) { return t == MXTRAIN_F32 ? 4 : 2; }

constexpr int64_t kMaxGroups = 65535;  // groups or matrices of one call

inline bool vec_c_ok(const void *c, int64_t ldc, int64_t stride_c, int type) {
  const int64_t v = 16 / size_of(type);
  return aligned(c, 16) && ldc % v == 0 && stride_c % v == 0;
}

}  // namespace mxt
