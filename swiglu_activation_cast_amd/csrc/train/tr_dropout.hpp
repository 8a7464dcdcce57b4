// tr_dropout.hpp -- dropout with a recomputed mask (gfx950).
//
//   y = residual + (r >= border ? x scale : 0),
//   border = p 65536, scale = 65536 / (65536 - border),
// where r are 16 bits of the Philox4x32-10 block of the element's eight
// columns (Salmon, Moraes, Dror and Shaw, 2011: ten rounds, each two 32 x 32 ->
// 64 bit products and four exclusive ors, with a key that grows by two constants).
//
// Bound by HBM: twenty products for eight elements stay below the time of their
// bytes, also without a residual.  (32 bits an element would double the products,
// and with them take longer than bf16's bytes.)  16384 x 8192 bf16 with the
// residual 127 us, 6.3 TB/s; without 97 us, 5.5 TB/s; 1021 x 2049 fp32 5 us.
#pragma once
#include "tr_rows.hpp"

namespace mxt {

struct DropArgs {
  const void *x, *res;
  void *y;
  int64_t ld_x, ld_res, ld_y;
  Pieces pieces;  // of 16 bytes
  u32 N, border;
  float scale;
  uint64_t seed, offset;
  const uint64_t *state;
};

__device__ __forceinline__ void philox(u32 (&c)[4], u32 k0, u32 k1) {
#pragma unroll
  for (int r = 0; r < 10; r++) {
    const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
    c[0] = (u32)(b >> 32) ^ c[1] ^ k0;
    c[1] = (u32)b;
    c[2] = (u32)(a >> 32) ^ c[3] ^ k1;
    c[3] = (u32)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// A piece is 16 bytes: eight bf16 columns and their block, or four fp32 ones and
// half of theirs (which the neighbouring lane computes too: as much of the
// generator for a byte).
template <class T, bool RES, bool NT>
__global__ __launch_bounds__(256) void k_dropout(const DropArgs a) {
  constexpr int VEC = 16 / (int)sizeof(T);
  uint64_t seed = a.seed, offset = a.offset;
  if (a.state) {
    seed += *gptr(a.state);
    offset += *gptr(a.state + 1);
  }
  for (int64_t first = (int64_t)blockIdx.x * 256; first < a.pieces.total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= a.pieces.total) continue;
    int64_t row;
    u32 piece;
    place_of(a.pieces, first, threadIdx.x, row, piece);
    const u32 col = piece * VEC;
    const int n = (int)min((u32)VEC, a.N - col);
    const T *px = static_cast<const T *>(a.x) + row * a.ld_x + col;
    const T *pr = RES ? static_cast<const T *>(a.res) + row * a.ld_res + col : nullptr;
    Piece<T, VEC> x, r;
    if (n == VEC) {
      x.template load<NT>(px);
      if constexpr (RES) r.template load<NT>(pr);
    } else {
      x.load(px, n);
      if constexpr (RES) r.load(pr, n);
    }
    u32 c[4] = {col / 8, (u32)row, (u32)offset, (u32)(offset >> 32)};
    philox(c, (u32)seed, (u32)(seed >> 32));
    if (VEC == 4 && piece % 2) {
      c[0] = c[2];
      c[1] = c[3];
    }
    float y[VEC];
#pragma unroll
    for (int i = 0; i < VEC; i++) {
      const u32 bits = i % 2 ? c[i / 2] >> 16 : c[i / 2] & 0xffffu;
      y[i] = bits >= a.border ? x.get(i) * a.scale : 0.0f;
      if constexpr (RES) y[i] += r.get(i);
    }
    x.set(y);
    T *py = static_cast<T *>(a.y) + row * a.ld_y + col;
    if (n == VEC) x.store(py);
    else x.store(py, 0, n);
  }
}

}  // namespace mxt
