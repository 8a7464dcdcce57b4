// tr_rows.hpp -- how the token operators walk rows: pieces of a row at any
// alignment, and the numbering of pieces.
#pragma once
#include "tr_common.hpp"

namespace mxt {

// Four words at an address that is only a multiple of two: the vector memory
// instructions take any address, so rows of odd widths and strides move 16 bytes
// at a time like others, and only a row's last piece can be short.
typedef u32 u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ u32x4_t load16(const void *p) {
  return *(const __attribute__((address_space(1))) u32x4_any *)p;  // (a template's argument would lose the alignment)
}
__device__ __forceinline__ void store16(void *p, u32x4_t v) { *(__attribute__((address_space(1))) u32x4_any *)p = v; }

// VEC elements of type T (uint16_t: bf16 bits) as they lie in memory.
template <class T, int VEC>
struct Piece {
  static constexpr int kWords = VEC * (int)sizeof(T) / 4;
  static_assert(kWords % 4 == 0, "whole 16-byte loads");
  u32 w[kWords];
  // The `n` first elements at p (n >= 1; zeros behind them).
  __device__ __forceinline__ void load(const T *p, int n) {
    if (n >= VEC) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const u32x4_t q = load16(reinterpret_cast<const u32 *>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; j++) w[i + j] = q[j];
      }
    } else {
      // without branches, so that the loads are in flight together
      T e[VEC - 1];
#pragma unroll
      for (int i = 0; i < VEC - 1; i++) e[i] = *gptr(p + min(i, n - 1));
      clear();
#pragma unroll
      for (int i = 0; i < VEC - 1; i++) {
        if constexpr (sizeof(T) == 4) w[i] = i < n ? __float_as_uint(e[i]) : 0;
        else w[i / 2] |= i < n ? (u32)e[i] << (i % 2 * 16) : 0;
      }
    }
  }
  __device__ __forceinline__ void store(T *p, int n) const {
    if (n >= VEC) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const u32x4_t q = {w[i], w[i + 1], w[i + 2], w[i + 3]};
        store16(reinterpret_cast<u32 *>(p) + i, q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC - 1; i++)
        if (i < n) {
          if constexpr (sizeof(T) == 4) *gptr(p + i) = __uint_as_float(w[i]);
          else *gptr(p + i) = (uint16_t)(w[i / 2] >> (i % 2 * 16));
        }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; i++) w[i] = 0;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return i % 2 ? mx::hi_f(w[i / 2]) : mx::lo_f(w[i / 2]);
  }
  __device__ __forceinline__ void set(const float *v) {
#pragma unroll
    for (int i = 0; i < kWords; i++) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = mx::pack_bf16(v[2 * i], v[2 * i + 1]);
    }
  }
};

// n / d for n < 2^31 and 1 <= d < 2^31: with 2^(l-1) < d <= 2^l and
// m = floor(2^(31+l) / d) + 1, m d exceeds 2^(31+l) by at most 2^l, so n m >> (31+l)
// is exact as long as n 2^l < 2^(31+l).  m <= 2^32 - 1 for every such d.
struct Divider {
  u32 d, m, shift;
  __device__ __forceinline__ u32 div(u32 n) const { return (u32)(((uint64_t)n * m) >> shift); }
};

inline Divider divider(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) l++;
  return {d, (u32)((1ull << (31 + l)) / d + 1), 31 + l};
}

// The pieces of a matrix's rows, numbered row by row.  A workgroup of 256
// threads takes 256 consecutive ones, the next workgroup's come after, and a grid
// smaller than the matrix goes round.
struct Pieces {
  int64_t total;  // rows x pieces of a row
  Divider per;    // pieces of a row
};

// The row of piece `first` + i (first wave-uniform, i < 2^30) and its number
// there.  A row has at most 2^29 pieces, so rest + i stays below 2^31; the
// 64-bit division is left to matrices of more pieces than that.
__device__ __forceinline__ void place_of(const Pieces &g, int64_t first, u32 i, int64_t &row, u32 &piece) {
  const int64_t row0 = g.total <= INT32_MAX ? 0 : first / g.per.d;
  const u32 rest = (u32)(first - row0 * g.per.d) + i, r = g.per.div(rest);
  row = row0 + r;
  piece = rest - r * g.per.d;
}

}  // namespace mxt
