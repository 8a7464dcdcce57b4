// tr_rows.hpp -- how the token operators walk rows: pieces of a row at any
// alignment, and the numbering of pieces.
#pragma once
#include "tr_common.hpp"

namespace mxt {

// Four words at an address that is only a multiple of two: the vector memory
// instructions take any address, so rows of odd widths and strides move 16 bytes
// at a time like others.
typedef u32 u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
// (Cast here rather than by gptr, whose template argument would lose the alignment.)
typedef __attribute__((address_space(1))) u32x4_any *glob16;
typedef const __attribute__((address_space(1))) u32x4_any *cglob16;

// VEC elements of type T (uint16_t: bf16 bits) as they lie in memory: 16 bytes'
// worth or more, or a single one.
template <class T, int VEC>
struct Piece {
  static constexpr int kWords = VEC == 1 ? 1 : VEC * (int)sizeof(T) / 4;
  static_assert(VEC == 1 || kWords % 4 == 0, "whole 16-byte loads");
  u32 w[kWords];
  template <bool NT = false>
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (VEC == 1) {
      put(0, *gptr(p));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const cglob16 from = (cglob16)(reinterpret_cast<const u32 *>(p) + i);
        const u32x4_t q = NT ? __builtin_nontemporal_load(from) : *from;
#pragma unroll
        for (int j = 0; j < 4; j++) w[i + j] = q[j];
      }
    }
  }
  // Past the caches (what is written here is larger than they are, or read next
  // by another XCD) where 16 bytes a lane fill whole lines; two such stores 32
  // bytes apart would each write half lines to memory.
  template <bool NT = true>
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (VEC == 1) {
      store(p, 0, 1);
    } else if constexpr (kWords == 4 && NT) {
      __builtin_nontemporal_store(u32x4_t{w[0], w[1], w[2], w[3]}, (glob16)p);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const u32x4_t q = {w[i], w[i + 1], w[i + 2], w[i + 3]};
        *(glob16)(reinterpret_cast<u32 *>(p) + i) = q;
      }
    }
  }
  // The n < VEC first elements (n >= 1), zeros behind them.  No branches between
  // the loads, so that they are in flight together.
  __device__ __forceinline__ void load(const T *p, int n) {
    T e[VEC];
#pragma unroll
    for (int i = 0; i < VEC - 1; i++) e[i] = *gptr(p + min(i, n - 1));
    clear();
#pragma unroll
    for (int i = 0; i < VEC - 1; i++)
      if (i < n) put(i, e[i]);
  }
  // Elements [from, to).
  __device__ __forceinline__ void store(T *p, int from, int to) const {
#pragma unroll
    for (int i = 0; i < VEC; i++)
      if (i >= from && i < to) {
        if constexpr (sizeof(T) == 4) *gptr(p + i) = __uint_as_float(w[i]);
        else *gptr(p + i) = (uint16_t)(w[i / 2] >> (i % 2 * 16));
      }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; i++) w[i] = 0;
  }
  // Element i, in a cleared place (or the first of its word).
  __device__ __forceinline__ void put(int i, T v) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v);
    else if (i % 2 == 0) w[i / 2] = v;
    else w[i / 2] |= (u32)v << 16;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return i % 2 ? mx::hi_f(w[i / 2]) : mx::lo_f(w[i / 2]);
  }
  __device__ __forceinline__ void set(const float *v) {
#pragma unroll
    for (int i = 0; i < kWords; i++) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = mx::pack_bf16(v[2 * i], VEC == 1 ? 0.0f : v[2 * i + 1]);
    }
  }
};

// First element of a row's piece.  Where a row of H elements (VEC or more) is not
// whole pieces, the last one starts VEC elements before the row's end and so
// shares elements with the one before: both compute and write the same values
// there.  Rows shorter than VEC are walked with VEC 1.
template <int VEC>
__device__ __forceinline__ u32 piece_col(u32 piece, u32 H) {
  return min(piece * VEC, H - VEC);
}

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
