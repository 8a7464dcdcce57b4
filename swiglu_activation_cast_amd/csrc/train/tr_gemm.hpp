// tr_gemm.hpp -- products of 16-bit matrices with fp32 sums on gfx950's matrix
// cores (v_mfma_f32_16x16x32_bf16 / _f16): the experts' products over ragged
// groups and the products of the Newton-Schulz steps.
//
//   C[m][n] = sum over k of A(m, k) B(n, k)
//
// Each operand is stored either with K adjacent (kKC: row m or n holds its
// K elements) or with its own index adjacent (kMC: row k holds the operand's
// M or N elements), so that the forward product (both kKC), the input
// gradient (B kMC) and the weight gradient (both kMC) read the tensors as they
// are, without a transposed copy.
//
// Structure: a 64 WI x 64 WJ tile of C per workgroup of four wavefronts
// (2 x 2, each 32 WI x 32 WJ, its sums in accumulation registers).  K is staged
// BK elements at a time in a ring of LDS slots that direct global -> LDS loads
// fill ahead of use.  A stage is consumed in steps of 32 (one MFMA deep):
// while a step's MFMAs run from registers, the next step's operands are read
// from LDS into the other register set, and the loads of a later stage are
// issued, between two MFMAs each.  The barrier of a stage sits before its last
// step's MFMAs, whose operands are then already in registers: from there the
// stage's slot is free to be filled again, and the MFMAs that follow cover the
// wait.  256 x 256 tiles with stages of 64 in a ring of two run fastest (8192 x
// 8192 x 8192, both kKC: 0.75 ms, 1.47 PFLOP/s; stages of 32 in a ring of four
// meet twice as many barriers, 8% slower; two workgroups to a CU with 128 x 256
// or 128 x 128 tiles read more of each operand, 20-35% slower).
//
// The card lowers its clock under such a product (1.7 to 1.95 GHz), so what an
// instruction moves counts beside what it takes: the 16x16x32 MFMA passes
// half as many accumulator bits through the registers per product as the
// 32x32x16 one, and is 4-6% faster here.
//
// LDS layouts.  kKC: rows of BK elements, 16-byte chunks at a position XORed
// with a function of the row, so that the 16 rows that a quarter of a
// wavefront reads at one chunk hit all banks once.  kMC: rows of the tile's
// 64 W columns, one per k; they are read with ds_read_b64_tr_b16, which
// hands lane i of 16 the i-th of 16 columns of four k rows (lane group of
// four = row; checked on gfx950); the chunk position is XORed with a function
// of k that spreads the eight k rows that half a wavefront reads over the
// banks.
//
// MFMA operand and result layout (16x16x32): lane l holds k 8 (l / 16) .. + 7
// of row l % 16; result register v of lane l is row 4 (l / 16) + v of the
// first operand, column l % 16 the second's row.  B is passed first, so that a
// lane holds four adjacent columns of one row of C (packed for the staged
// store at the end).
#pragma once
#include <type_traits>

#include "tr_common.hpp"

namespace mxt {

// Loads [FROM, TO) of a stage.
template <int FROM, int TO>
struct Part {
  static constexpr int from = FROM, to = TO;
};

enum Layout { kKC = 0, kMC = 1 };
enum Mode { kGroupM = 1, kGroupK = 2 };
enum Elem { kBf16 = 0, kF16 = 1 };

constexpr int kThreads = 256;
constexpr int kTileRows = 16;             // tile rows per band of the tile order
constexpr int64_t kMaxLd = int64_t(1) << 22;  // 255 rows of as many elements and 512 bytes of the next stay below 2^31 bytes

struct GemmArgs {
  const uint16_t *a, *b;
  int64_t lda, ldb;
  int64_t stride_a, stride_b;  // per batch entry; stride_b per expert in kGroupM
  int64_t M, N, K;             // M: all rows in kGroupM; K: all of it in kGroupK
  void *c;
  int64_t ldc, stride_c;       // stride_c per batch entry or group
  const int32_t *ends;         // cumulative group ends (device), G of them
  int32_t G;                   // groups, or batch entries
  int32_t tiles_m, tiles_n;    // tiles_m: an upper bound in kGroupM
  int32_t vec_c;               // whole 16-byte chunks of C may be stored
  int32_t cus;                 // compute units (see work_item)
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef u32 u32x2_t __attribute__((ext_vector_type(2)));

#define MXT_LDS __attribute__((address_space(3)))

// f(0), f(1), ... f(N - 1), each with its index as a compile-time constant.
template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// 16 bytes a lane, global -> LDS: lane l's land at LDS byte lds + AT + 16 l.
// Asm, so that the compiler does not wait for it before LDS reads of other
// slots; wait_vm awaits it.  M0 takes the LDS base, which needs one wait state
// between its write and the load; nothing else in these kernels uses M0, so it
// is not put back.  Three instructions, since a wavefront alone on its SIMD
// has room for about seven between two MFMAs (with the base's sum, M0 put back
// and the bounds select per load, ten, a stage took 2650 cycles for its 2048
// of MFMA).
template <int AT>
__device__ __forceinline__ void dma16(const void *base, u32 off, u32 lds) {
  asm volatile(
      "s_add_u32 m0, %0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2" ::"s"(lds),
      "v"(off), "s"(base), "n"(AT)
      : "scc");
}
// A value that every lane holds alike, in a scalar register.
template <class P>
__device__ __forceinline__ P *uniform(P *p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  return (P *)(uintptr_t)(((uint64_t)(u32)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
                          (u32)__builtin_amdgcn_readfirstlane((int)(u32)v));
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ u32 lds_addr(const void *p) { return (u32)(uintptr_t)(const MXT_LDS void *)p; }

template <int EL>
__device__ __forceinline__ f32x4_t mfma(u32x4_t first, u32x4_t second, f32x4_t c) {
  typedef __bf16 b8 __attribute__((ext_vector_type(8)));
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  if constexpr (EL == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, first), __builtin_bit_cast(b8, second), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, first), __builtin_bit_cast(h8, second), c, 0, 0, 0);
}

// One operand of a tile: W 64-row halves (64 W rows of the operand, or
// columns where it is stored kMC).  `rows` of them exist (>= 1); the others
// are read as the last one and never stored.  A wavefront fills kLoads
// kilobytes of each stage.
template <int L, int W, int BK>
struct Operand {
  static constexpr int kBK = BK, kKS = BK / 32;  // elements and MFMA steps of a stage
  static constexpr int kRows = 64 * W;
  static constexpr int kBytes = kRows * kBK * 2;  // of a stage
  static constexpr int kLoads = kBytes / 1024 / 4;
  static constexpr int kRowB = L == kKC ? kBK * 2 : kRows * 2;  // bytes of an LDS row
  static constexpr int kPer = 1024 / kRowB;                     // LDS rows per load
  static constexpr int kLanes = 64 / kPer;                      // lanes (chunks) per LDS row

  const uint8_t *base;  // of the tile's first k (uniform)
  int64_t step;         // bytes from a stage to the next (uniform)
  u32 off[kLoads];      // this lane's byte offset in each load
  u32 tail[kLoads];     // the same at the stage's first k
  u32 cur[kLoads];      // which of the two the loads use
  int k_of[kLoads];     // first k (within the stage) of what the lane loads
  u32 lds_w;            // LDS byte (within a stage's operand) of this wavefront's first load
  u32 rd[L == kKC ? kKS : 2 * W];  // this lane's LDS read offsets

  // XOR of the chunk position in LDS row r.  A 16-byte read serves lanes 0-3,
  // 12-15 and 20-27 at once, then 4-11, 16-19 and 28-31: with four chunks to a
  // row, rows 4 a .. 4 a + 3 of the first chunk at a = 0 and 3 meet those of the
  // second at a = 1 and 2, which XOR by -a keeps apart (by a, half of all reads
  // conflicted).
  static __device__ __forceinline__ u32 key(u32 r) {
    if constexpr (L == kKC && BK == 64) return (r >> 1) & 7u;
    else if constexpr (L == kKC) return (0u - (r >> 2)) & 3u;
    else if constexpr (W == 1) return (((r >> 1) & 1u) | ((r >> 3) & 1u) << 1) << 1;  // 128-byte rows: two per turn of the banks
    else return ((r & 3u) | ((r >> 3) & 1u) << 2) << 1;
  }

  // `blk0` + x * `blk_step` is the x-th 32-row block of this wavefront.
  __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, u32 rows, int wave, int lane, int blk0,
                                       int blk_step) {
    base = uniform(reinterpret_cast<const uint8_t *>(p));
    step = L == kKC ? (int64_t)kBK * 2 : (int64_t)kBK * ld * 2;
    lds_w = (u32)(wave * kLoads) * 1024u;
#pragma unroll
    for (int q = 0; q < kLoads; q++) {
      const u32 r = (u32)((wave * kLoads + q) * kPer) + (u32)lane / kLanes;  // LDS row
      const u32 c = ((u32)lane % kLanes) ^ key(r);                          // chunk of that row
      if constexpr (L == kKC) {
        off[q] = min(r, rows - 1) * (u32)(ld * 2) + c * 16u;
        tail[q] = min(r, rows - 1) * (u32)(ld * 2);
        k_of[q] = (int)c * 8;
      } else {
        const u32 cc = min(c, (rows - 1) / 8u) * 16u;
        off[q] = r * (u32)(ld * 2) + cc;
        tail[q] = cc;
        k_of[q] = (int)r;
      }
    }
    const u32 gq = (u32)lane >> 4, i = (u32)lane & 15u;
    if constexpr (L == kKC) {
#pragma unroll
      for (int s = 0; s < kKS; s++) rd[s] = ((u32)blk0 * 32u + i) * kRowB + ((((u32)(4 * s) + gq) ^ key(i)) << 4);
    } else {
      const u32 k = 8u * gq + (i >> 2);  // of a step; key(k) is the same for every step and half
#pragma unroll
      for (int x = 0; x < 2 * W; x++) {
        const u32 chunk = (u32)(blk0 + x / 2 * blk_step) * 4u + 2u * (u32)(x & 1) + ((i & 3u) >> 1);
        rd[x] = k * kRowB + ((chunk ^ key(k)) << 4) + (i & 1u) * 8u;
      }
    }
  }
  // From here on the stages to be loaded have kmax elements of K: chunks (rows)
  // at or past it are read at the stage's first k instead, and cleared once
  // they have landed.
  __device__ __forceinline__ void set_kmax(int kmax) {
#pragma unroll
    for (int q = 0; q < kLoads; q++) cur[q] = k_of[q] < kmax ? off[q] : tail[q];
  }
  // Load number Q of the stage at `src`, AT bytes past `slot`, this wavefront's
  // first byte.
  template <int Q, int AT>
  __device__ __forceinline__ void load(const uint8_t *src, u32 slot) const {
    dma16<AT + Q * 1024>(src, cur[Q], slot);
  }
  // This lane's part of a landed stage, k >= kmax -> 0.
  __device__ __forceinline__ void clear(MXT_LDS uint8_t *slot, int lane, int kmax) const {
#pragma unroll
    for (int q = 0; q < kLoads; q++) {
      MXT_LDS u32x4_t *p = (MXT_LDS u32x4_t *)(slot + lds_w + (u32)q * 1024u + 16u * (u32)lane);
      if constexpr (L == kMC) {
        if (k_of[q] >= kmax) *p = u32x4_t{0, 0, 0, 0};
      } else if (k_of[q] + 8 > kmax) {
        const int keep = kmax - k_of[q];  // elements of the chunk that exist
        u32x4_t v = *p;
#pragma unroll
        for (int d = 0; d < 4; d++) v[d] &= keep >= 2 * d + 2 ? 0xffffffffu : keep == 2 * d + 1 ? 0xffffu : 0u;
        *p = v;
      }
    }
  }
  static constexpr int kReads = L == kKC ? 2 * W : 4 * W;  // LDS reads of a step
  // Read number t of step s into the fragments.
  __device__ __forceinline__ void read(const MXT_LDS uint8_t *slot, int s, int t, int blk_step, u32x4_t *f) const {
    if constexpr (L == kKC) {
      f[t] = *(const MXT_LDS u32x4_t *)(slot + rd[s] + (u32)((t / 2) * blk_step * 32 + (t & 1) * 16) * kRowB);
    } else {
      const int x = t / 2, j = t % 2;
      const u32x2_t v = __builtin_bit_cast(
          u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((MXT_LDS s16x4_t *)(slot + rd[x] + (u32)(32 * s + 4 * j) * kRowB)));
      f[x][2 * j] = v[0];
      f[x][2 * j + 1] = v[1];
    }
  }
};

// What a tile's workgroup computes: `rows` x `cols` of C over `k_len` of K from
// the operands' bases.  With SPLIT, A and B each come as a high and a low plane
// and the sum runs over high x low, high x high and low x high.  With TWICE, K is
// gone through twice where `passes` is 2: over a_lo and b_lo, then over a and b
// (an operand of one plane gives it as both), so that one operand's low plane
// enters with no other change to a stage.
struct Tile {
  const uint16_t *a, *b;        // at the tile's first row (column) and k
  const uint16_t *a_lo, *b_lo;  // SPLIT, TWICE
  int64_t k_len;
  u32 rows, cols;
  u32 first;                    // any number: which stage of K (modulo them) comes first (not with TWICE)
  int32_t passes;               // TWICE: 1 or 2
};

template <int EL, int AL, int BL, int WI, int WJ, int BK, int RING, bool SPLIT, bool TWICE = false, class Emit>
__device__ __forceinline__ void gemm_tile(const GemmArgs &g, const Tile &t, uint8_t *smem, const Emit &emit) {
  using A = Operand<AL, WI, BK>;
  using B = Operand<BL, WJ, BK>;
  constexpr int kBK = BK, kKS = BK / 32, kPl = SPLIT ? 2 : 1;
  // a slot: A's planes, then B's
  constexpr int kSlotB = kPl * A::kBytes, kSlot = kSlotB + kPl * B::kBytes;
  constexpr int kLoads = kPl * (A::kLoads + B::kLoads);
  static_assert((RING - 1) * kLoads < 64, "the count that wait_vm can hold");
  constexpr int WA = 2 * WI, WB = 2 * WJ;  // 16-row blocks
  constexpr int kMfmas = WA * WB;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1;
  // 32-row blocks of C: A's alternate between the two wavefront rows (a short
  // tile has rows in both), B's are adjacent
  A oa;
  B ob;
  oa.init(t.a, g.lda, t.rows, w, lane, wm, 2);
  ob.init(t.b, g.ldb, t.cols, w, lane, WJ * wn, 1);

  f32x4_t acc[WA][WB];
#pragma unroll
  for (int i = 0; i < WA; i++)
#pragma unroll
    for (int j = 0; j < WB; j++) acc[i][j] = f32x4_t{};

  static_assert(!(SPLIT && TWICE), "two ways to take a low plane");
  const int n_pass = __builtin_amdgcn_readfirstlane((int)((t.k_len + kBK - 1) / kBK));  // stages of K
  const int n_stage = TWICE ? n_pass * __builtin_amdgcn_readfirstlane(t.passes) : n_pass;
  const int k_tail = (int)(t.k_len - (int64_t)(n_pass - 1) * kBK);  // k in K's last stage, 1 .. kBK
  MXT_LDS uint8_t *lds = (MXT_LDS uint8_t *)smem;
  const u32 lds0 = lds_addr(smem);

  const uint8_t *a_lo = nullptr, *b_lo = nullptr;
  if constexpr (SPLIT || TWICE) {
    a_lo = uniform(reinterpret_cast<const uint8_t *>(t.a_lo));
    b_lo = uniform(reinterpret_cast<const uint8_t *>(t.b_lo));
  }
  struct Src {
    const uint8_t *a[2], *b[2];  // the stage in each plane
    u32 slot_a, slot_b;          // where this wavefront's first load of an operand lands
  };
  int kmax = kBK;  // of the stages being loaded
  oa.set_kmax(kmax);
  ob.set_kmax(kmax);
  // The stages of K in turn, from t.first on; with TWICE, the last n_pass of them
  // are the high planes'.
  const int rot = !TWICE && n_stage > 0 ? __builtin_amdgcn_readfirstlane((int)(t.first % (u32)n_stage)) : 0;
  auto high = [&](int st) { return !TWICE || st >= n_stage - n_pass; };
  auto place = [&](int st) {
    if constexpr (TWICE) return high(st) ? st - (n_stage - n_pass) : st;
    else return st + rot < n_stage ? st + rot : st + rot - n_stage;
  };
  // Stages past the last re-read it into a slot that is not read again.
  auto source = [&](int st) {
    const int at = min(st, n_stage - 1), s = place(at);
    Src r;
    r.a[0] = (high(at) ? oa.base : a_lo) + s * oa.step;
    r.b[0] = (high(at) ? ob.base : b_lo) + s * ob.step;
    r.a[1] = SPLIT ? a_lo + s * oa.step : nullptr;
    r.b[1] = SPLIT ? b_lo + s * ob.step : nullptr;
    r.slot_a = lds0 + (u32)(st % RING) * kSlot + oa.lds_w;
    r.slot_b = lds0 + (u32)(st % RING) * kSlot + kSlotB + ob.lds_w;
    const int k = s == n_pass - 1 ? k_tail : kBK;
    if (k != kmax) {  // uniform; only around a partial last stage
      kmax = k;
      oa.set_kmax(k);
      ob.set_kmax(k);
    }
    return r;
  };
  auto load = [&](auto q, const Src &r) {
    constexpr int Q = decltype(q)::value, P = Q / (A::kLoads + B::kLoads), R = Q % (A::kLoads + B::kLoads);
    if constexpr (R < A::kLoads) oa.template load<R, P * A::kBytes>(r.a[P], r.slot_a);
    else ob.template load<R - A::kLoads, P * B::kBytes>(r.b[P], r.slot_b);
  };
  // Stage st has landed: clear what lies past K (each lane what it loaded).
  auto clear = [&](int st) {
    if (k_tail == kBK || st >= n_stage || place(st) != n_pass - 1) return;
    MXT_LDS uint8_t *slot = lds + (st % RING) * kSlot;
#pragma unroll
    for (int p = 0; p < kPl; p++) {
      oa.clear(slot + p * A::kBytes, lane, k_tail);
      ob.clear(slot + kSlotB + p * B::kBytes, lane, k_tail);
    }
  };

  using Yes = std::true_type;
  using No = std::false_type;
  // MFMAs of one step, a times b; between them `n_reads` LDS reads, after every
  // other MFMA while there are enough, and, where asked, all loads of a stage,
  // spread evenly.  (Loads over the whole stage leave the last of them too
  // little time to land, 10% slower; packed more densely they queue, 5%.)
  auto phase = [&](auto do_mfma, auto loads, auto n_reads, u32x4_t *fa, u32x4_t *fb, const Src &src, auto &&read) {
    constexpr int q0 = decltype(loads)::from, Q = decltype(loads)::to - q0, R = decltype(n_reads)::value;
    constexpr int kEvery = R * 2 <= kMfmas ? 2 : 1, kPer = (R + kMfmas - 1) / kMfmas;
    static_for<kMfmas>([&](auto kk) {
      constexpr int k = decltype(kk)::value, i = k / WB, j = k % WB;
      if constexpr (decltype(do_mfma)::value) acc[i][j] = mfma<EL>(fb[j], fa[i], acc[i][j]);
      if constexpr (k % kEvery == 0) {
#pragma unroll
        for (int n = k / kEvery * kPer; n < (k / kEvery + 1) * kPer; n++)
          if (n < R) read(n);
      }
      static_for<(k + 1) * Q / kMfmas - k * Q / kMfmas>(
          [&](auto q) { load(std::integral_constant<int, q0 + k * Q / kMfmas + decltype(q)::value>{}, src); });
      __builtin_amdgcn_sched_barrier(0);  // keep this order
    });
  };
  // LDS read number n of A and B of step s of a slot, in the order in which the
  // MFMAs need them: A's first block, B's blocks, A's others.
  constexpr int kA1 = A::kReads / WA;  // reads of one A block
  auto read_ab = [&](const MXT_LDS uint8_t *slot_a, const MXT_LDS uint8_t *slot_b, int s, int n, u32x4_t *fa, u32x4_t *fb) {
    if (n < kA1) oa.read(slot_a, s, n, 2, fa);
    else if (n < kA1 + B::kReads) ob.read(slot_b, s, n - kA1, 1, fb);
    else oa.read(slot_a, s, n - B::kReads, 2, fa);
  };
  using NA = std::integral_constant<int, A::kReads>;
  using NB = std::integral_constant<int, B::kReads>;
  using NAB = std::integral_constant<int, A::kReads + B::kReads>;

  // Fragments: [0], [1] are the two steps in turn, or with SPLIT the high and
  // low planes of one step.
  u32x4_t fa[2][WA], fb[2][WB];
  static_assert(SPLIT || kKS % 2 == 0, "the last step of a stage leaves its operands in [1]");
  // Stage st: the last MFMAs of stage st - 1, whose operands are in registers,
  // then its own but the last, whose operands it leaves there.  At its end
  // stage st + 1 has landed and stage st's slot is free.
  auto stage = [&](auto has_last, int st) {
    const MXT_LDS uint8_t *slot = lds + (st % RING) * kSlot;
    constexpr bool first = !decltype(has_last)::value;
    constexpr int kAll = first ? 0 : kLoads;
    constexpr int kCut = kAll * 2 / 3;  // SPLIT, whose phases are longer: two thirds in the first, the rest in the second
    // the loads of the stage that takes over stage st - 1's slot
    const Src src = first ? Src{} : source(st - 1 + RING);
    if constexpr (SPLIT) {
      // low x high of the step before while high A and low B are read, then
      // high x low (reading high B) and high x high (reading low A): three
      // phases on one set of registers
#pragma unroll
      for (int s = 0; s < kKS; s++) {
        auto rd = [&](int n) { read_ab(slot, slot + kSlotB + B::kBytes, s, n, fa[0], fb[1]); };
        auto rdb = [&](int n) { ob.read(slot + kSlotB, s, n, 1, fb[0]); };
        if (s == 0) phase(has_last, Part<0, kCut>{}, NAB{}, fa[1], fb[0], src, rd);
        else phase(Yes{}, Part<0, 0>{}, NAB{}, fa[1], fb[0], src, rd);
        if (s == 0) phase(Yes{}, Part<kCut, kAll>{}, NB{}, fa[0], fb[1], src, rdb);
        else phase(Yes{}, Part<0, 0>{}, NB{}, fa[0], fb[1], src, rdb);
        phase(Yes{}, Part<0, 0>{}, NA{}, fa[0], fb[0], src, [&](int n) { oa.read(slot + A::kBytes, s, n, 2, fa[1]); });
      }
    } else {
      phase(has_last, Part<0, kAll>{}, NAB{}, fa[1], fb[1], src, [&](int n) { read_ab(slot, slot + kSlotB, 0, n, fa[0], fb[0]); });
#pragma unroll
      for (int s = 1; s < kKS; s++)
        phase(Yes{}, Part<0, 0>{}, NAB{}, fa[(s + 1) & 1], fb[(s + 1) & 1], src,
              [&](int n) { read_ab(slot, slot + kSlotB, s, n, fa[s & 1], fb[s & 1]); });
    }
#if __HIP_DEVICE_COMPILE__
    // keep this stage's results in its block
#pragma unroll
    for (int i = 0; i < WA; i++) {
#pragma unroll
      for (int j = 0; j < WB; j++) asm volatile("" ::"a"(acc[i][j]));
      asm volatile("" ::"v"(fa[1][i]));
    }
#pragma unroll
    for (int j = 0; j < WB; j++) asm volatile("" ::"v"(fb[SPLIT ? 0 : 1][j]));
#endif
    // issued so far: stages up to st - 1 + RING
    wait_vm<(RING - 2) * kLoads>();
    clear(st + 1);
    __syncthreads();
  };

  if (n_stage > 0) {
#pragma unroll
    for (int st = 0; st < RING; st++) {
      const Src src = source(st);
      static_for<kLoads>([&](auto q) { load(q, src); });
    }
    wait_vm<(RING - 1) * kLoads>();
    clear(0);
    __syncthreads();
    stage(No{}, 0);
    for (int st = 1; st < n_stage; st++) stage(Yes{}, st);
    constexpr int last_b = SPLIT ? 0 : 1;
#pragma unroll
    for (int k = 0; k < kMfmas; k++) acc[k / WB][k % WB] = mfma<EL>(fb[last_b][k % WB], fa[1][k / WB], acc[k / WB][k % WB]);
    wait_vm<0>();  // nothing may still be landing in LDS when the workgroup ends or goes on
  }

  // The results: a lane holds four adjacent columns of one row, rows across the
  // lanes, which stored as they are would touch 32 rows of C 16 bytes at a
  // time (measured: 430 us of a 570 us product of 8192 x 8192 x 1024).  So each
  // wavefront passes them through LDS of its own, one 32-row block after
  // another, and stores whole rows of its block.
  __syncthreads();  // no load is in flight and no operand read is left: LDS is free
  constexpr int kChunks = (Emit::kF32 ? 8 : 4) * WJ;  // 16-byte chunks of a staged row
  constexpr int kRow = kChunks * 16, kPlane = 32 * kRow;
  constexpr int kTurn = kChunks >= 16 ? 1 : 16 / kChunks;  // staged rows per turn of the banks
  static_assert(4 * Emit::kPlanes * kPlane <= RING * kSlot, "the staged blocks fit the slots");
  MXT_LDS uint8_t *mine = lds + w * (Emit::kPlanes * kPlane);
  auto chunk_at = [&](u32 row, u32 c) { return row * kRow + ((c ^ ((row / kTurn) & (kChunks - 1))) << 4); };
  const u32 h = (u32)lane >> 4, r16 = (u32)lane & 15u;
  const u32 nw = 32u * (u32)(WJ * wn);  // the wavefront's first column
#pragma unroll
  for (int i = 0; i < WI; i++) {
    const u32 mb = 32u * (u32)(2 * i + wm);
    if (mb >= t.rows) break;  // uniform
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < WB; j++)
#pragma unroll
      for (int q = 0; q < 2; q++) {
        const f32x4_t v = acc[2 * i + q][j];
        const u32 r = r16 + 16u * (u32)q;
        const u32 n = 16u * (u32)j + 4u * h;
        if constexpr (Emit::kF32) {
          *(MXT_LDS f32x4_t *)(mine + chunk_at(r, n / 4)) = emit.map(mb + r, nw + n, v);
        } else {
          u32x2_t p[Emit::kPlanes];
          emit.pack(mb + r, nw + n, v, p);
#pragma unroll
          for (int k = 0; k < Emit::kPlanes; k++)
            *(MXT_LDS u32x2_t *)(mine + k * kPlane + chunk_at(r, n / 8) + (n & 4u) * 2) = p[k];
        }
      }
    asm volatile("" ::: "memory");  // the wavefront's LDS operations run in order: no wait is needed
#pragma unroll
    for (int k = 0; k < Emit::kPlanes; k++) {
#pragma unroll
      for (int it = 0; it < kChunks / 2; it++) {
        const u32 at = (u32)it * 64u + (u32)lane, row = at / kChunks, c = at % kChunks;
        const u32x4_t v = *(const MXT_LDS u32x4_t *)(mine + k * kPlane + chunk_at(row, c));
        const u32 n = nw + c * (Emit::kF32 ? 4u : 8u);
        if (mb + row < t.rows && n < t.cols) emit.store(k, mb + row, n, v);
      }
      if constexpr (Emit::kMirror) {
        // the transposed block: a transpose read gives a lane four rows of one
        // column, two of them the eight that it stores
        if (emit.mirrored()) {
          const u32 li = (u32)lane & 15u, lg = (u32)lane >> 4;
#pragma unroll
          for (int it = 0; it < 2 * WJ; it++) {  // 16 columns; lane group lg takes rows 8 lg .. + 7
            u32x4_t v;
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const u32 row = 8u * lg + 4u * (u32)e + (li >> 2), n = 16u * (u32)it + 4u * (li & 3u);
              const u32x2_t q = __builtin_bit_cast(
                  u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                               (MXT_LDS s16x4_t *)(mine + k * kPlane + chunk_at(row, n / 8) + (n & 4u) * 2)));
              v[2 * e] = q[0];
              v[2 * e + 1] = q[1];
            }
            const u32 n = nw + 16u * (u32)it + li, m = mb + 8u * lg;
            if (m < t.rows && n < t.cols) emit.store_mirror(k, n, m, v);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------- the experts' products
// Results of a tile at c (row stride ldc), fp32 or rounded to bf16.
template <bool F32>
struct EmitC {
  static constexpr bool kF32 = F32, kMirror = false;
  static constexpr int kPlanes = 1;
  void *c;
  int64_t ldc;
  u32 cols;
  bool vec;  // whole 16-byte chunks of C may be stored
  __device__ __forceinline__ f32x4_t map(u32, u32, f32x4_t v) const { return v; }
  __device__ __forceinline__ void pack(u32, u32, f32x4_t v, u32x2_t *p) const {
    p[0] = u32x2_t{mx::pack_bf16(v[0], v[1]), mx::pack_bf16(v[2], v[3])};
  }
  __device__ __forceinline__ void store(int, u32 m, u32 n, u32x4_t v) const {
    constexpr u32 N = F32 ? 4 : 8;
    uint8_t *p = static_cast<uint8_t *>(c) + ((int64_t)m * ldc + n) * (F32 ? 4 : 2);
    if (vec && n + N <= cols) {
      *gptr(reinterpret_cast<u32x4_t *>(p)) = v;
    } else {
#pragma unroll
      for (u32 e = 0; e < N; e++)
        if (n + e < cols) {
          if constexpr (F32) *gptr(reinterpret_cast<u32 *>(p) + e) = v[e];
          else *gptr(reinterpret_cast<uint16_t *>(p) + e) = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
        }
    }
  }
};

// Group bounds: cumulative ends, made non-decreasing and clamped into [0, M]:
// any values give ranges inside the matrices.
//
// kGroupM: the group and first row of tile row `want` (tile rows of BM rows,
// counted group by group from each group's first row), and the number of tile
// rows.  64 groups a time, one per lane: a running maximum (the clamp) and a
// running sum of tile counts over the lanes.
struct GroupTile {
  int32_t group;  // -1: past the last
  int64_t m0, m_end, total;
};
template <int BM>
__device__ __forceinline__ GroupTile find_tile(const int32_t *ends, int32_t G, int64_t M, int64_t want) {
  const int lane = threadIdx.x & 63;
  GroupTile r{-1, 0, 0, 0};
  int32_t floor_end = 0;
  int64_t before = 0;
  for (int32_t g0 = 0; g0 < G; g0 += 64) {
    const int32_t m32 = (int32_t)M;
    int32_t end = g0 + lane < G ? min(max(*gptr(ends + g0 + lane), 0), m32) : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t up = __shfl_up(end, o, 64);
      if (lane >= o) end = max(end, up);
    }
    end = max(end, floor_end);
    int32_t start = __shfl_up(end, 1, 64);
    if (lane == 0) start = floor_end;
    int32_t tiles = (end - start + BM - 1) / BM, sum = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t up = __shfl_up(sum, o, 64);
      if (lane >= o) sum += up;
    }
    const uint64_t hit = __ballot(want < before + sum);
    if (hit && r.group < 0) {
      const int e = __builtin_amdgcn_readfirstlane((int)__ffsll((unsigned long long)hit) - 1);
      r.group = g0 + e;
      const int32_t s = __builtin_amdgcn_readlane(start, e), inc = __builtin_amdgcn_readlane(sum, e);
      const int32_t own = __builtin_amdgcn_readlane(tiles, e);
      r.m0 = s + (int64_t)((int32_t)(want - before) - (inc - own)) * BM;
      r.m_end = __builtin_amdgcn_readlane(end, e);
    }
    floor_end = __builtin_amdgcn_readlane(end, 63);
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  r.total = before;
  return r;
}

// kGroupK: the start and end of group `want`.
__device__ __forceinline__ void find_group(const int32_t *ends, int32_t want, int64_t T, int64_t &start, int64_t &end) {
  const int lane = threadIdx.x & 63;
  int32_t below = 0;  // largest end before `want`
  for (int32_t e = lane; e < want; e += 64) below = max(below, *gptr(ends + e));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) below = max(below, __shfl_xor(below, o, 64));
  below = __builtin_amdgcn_readfirstlane(below);
  start = min<int64_t>(below, T);
  end = min<int64_t>(max(below, __builtin_amdgcn_readfirstlane(*gptr(ends + want))), T);
}

// Position in the tile order -> tile row and column: bands of kTileRows tile
// rows, walked column by column.
__device__ __forceinline__ void tile_of(u32 L, u32 tiles_m, u32 tiles_n, u32 &tm, u32 &tn) {
  const u32 per = (u32)kTileRows * tiles_n, band = L / per, in = L % per;
  const u32 rows = min((u32)kTileRows, tiles_m - band * (u32)kTileRows);
  tm = band * (u32)kTileRows + in % rows;
  tn = in / rows;
}
// Work item -> position.  256 positions of a band are a square of 16 x 16
// tiles, which the 256 CUs compute together; workgroups are dealt to the 8 XCDs
// in turn, and each XCD takes a 4 x 8 part of the square, so that its L2
// serves 12 operand tiles for 32 results and all of them together read 32 for
// 256.  (Each XCD going through an eighth of all tiles by itself reads up to
// 96, and of four experts' weights at once: 10% slower at 16384 tokens over
// four experts of 8192 x 5120.)  Positions past the last whole square stay.
__device__ __forceinline__ u32 square_order(u32 b, u32 whole) {
  if (b >= (whole & ~255u)) return b;
  const u32 x = b & 7u, j = (b >> 3) & 31u;
  const u32 row = 4u * (x & 3u) + (j & 3u), col = 8u * (x >> 2) + (j >> 2);
  return (b & ~255u) + col * 16u + row;
}

// A launch of R tiles of 256 x 256, one to a CU at a time, runs in rounds of
// `cus`.  If the tiles of a last partial round would leave at least half of
// the CUs idle, they run as 256 x 128 halves, if at least three quarters, as
// 256 x 64 quarters, so that the round ends in a little over half (a quarter)
// of the time.  item -> tile index, and which of its `parts`; false: no work.
struct Item {
  u32 L, part, parts;
};
__device__ __forceinline__ bool work_item(u32 b, u32 R, u32 cus, Item &it) {
  const u32 tail = R % cus, R0 = R - tail;
  it.parts = 1;
  it.part = 0;
  if (b < R0) {
    it.L = b;
    return true;
  }
  it.parts = tail <= cus / 4 ? 4u : tail <= cus / 2 ? 2u : 1u;
  it.L = R0 + (b - R0) / it.parts;
  it.part = (b - R0) % it.parts;
  return it.L < R;
}
// Work items of R tiles, and an upper bound over all R' <= R.
inline int64_t work_items(int64_t R, int64_t cus) {
  const int64_t tail = R % cus;
  return R + (tail <= cus / 4 ? 3 * tail : tail <= cus / 2 ? tail : 0);
}
inline int64_t work_items_bound(int64_t R, int64_t cus) {
  const int64_t extra = 3 * (cus / 4) > cus / 2 ? 3 * (cus / 4) : cus / 2;
  return R + extra;
}

// WI = WJ = 4: 256 x 256 tiles, short ones (a group's last rows) and those of a
// last partial round cut down; smaller tiles, two workgroups to a CU.
template <int MODE, int AL, int BL, int WI, int WJ, int BK, int RING, bool F32>
__global__ __launch_bounds__(kThreads, WI * WJ > 8 ? 1 : 2) void k_group_gemm(const GemmArgs g) {
  constexpr int BM = 64 * WI, BN = 64 * WJ;
  constexpr bool kBig = WI == 4 && WJ == 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING * (BM + BN) * BK * 2];
  Tile t{};
  u32 tm, tn;
  Item it{blockIdx.x, 0, 1};
  EmitC<F32> emit{g.c, g.ldc, 0, g.vec_c != 0};
  if constexpr (MODE == kGroupM) {
    // the real number of tile rows first, then this workgroup's tile
    const u32 total = (u32)find_tile<BM>(g.ends, g.G, g.M, INT64_MAX).total;
    const u32 R = total * (u32)g.tiles_n;
    if (kBig ? !work_item(blockIdx.x, R, (u32)g.cus, it) : blockIdx.x >= R) return;
    const u32 whole = kBig ? R - R % (u32)g.cus : R;
    tile_of(square_order(it.L, whole), total, (u32)g.tiles_n, tm, tn);
    const GroupTile gt = find_tile<BM>(g.ends, g.G, g.M, tm);
    t.a = g.a + gt.m0 * g.lda;
    t.b = g.b + (int64_t)gt.group * g.stride_b;
    t.rows = (u32)min<int64_t>(BM, gt.m_end - gt.m0);
    t.k_len = g.K;
    emit.c = F32 ? (void *)(static_cast<float *>(g.c) + gt.m0 * g.ldc) : (void *)(static_cast<uint16_t *>(g.c) + gt.m0 * g.ldc);
  } else {
    // the groups one after another
    const u32 per = (u32)g.tiles_m * (u32)g.tiles_n, R = per * (u32)g.G;
    if (kBig && !work_item(blockIdx.x, R, (u32)g.cus, it)) return;
    const u32 whole = kBig ? R - R % (u32)g.cus : R;
    const u32 L = square_order(it.L, whole);
    const int32_t grp = (int32_t)(L / per);
    tile_of(L % per, (u32)g.tiles_m, (u32)g.tiles_n, tm, tn);
    int64_t start, end;
    find_group(g.ends, grp, g.K, start, end);
    const int64_t m0 = (int64_t)tm * BM;
    t.a = g.a + start * g.lda + m0;
    t.b = g.b + start * g.ldb;
    t.rows = (u32)min<int64_t>(BM, g.M - m0);
    t.k_len = end - start;
    const int64_t at = (int64_t)grp * g.stride_c + m0 * g.ldc;
    emit.c = F32 ? (void *)(static_cast<float *>(g.c) + at) : (void *)(static_cast<uint16_t *>(g.c) + at);
  }
  const int64_t n0 = (int64_t)tn * BN + it.part * (BN / it.parts);
  if (n0 >= g.N) return;  // a part past the last column
  t.b += BL == kKC ? n0 * g.ldb : n0;
  t.cols = emit.cols = (u32)min<int64_t>(BN / it.parts, g.N - n0);
  emit.c = F32 ? (void *)(static_cast<float *>(emit.c) + n0) : (void *)(static_cast<uint16_t *>(emit.c) + n0);
  // Tiles of few rows stream the weights, each its own rows of them, and where
  // those are a power of two apart, tiles that go through K in step read from
  // few of the memory channels at a time.  So each starts at another stage (24
  // tokens over 16 experts, 4096 x 2048: 55 -> 41 us, 5.2 TB/s).
  if (WI == 1 && BL == kKC) t.first = blockIdx.x;
  if constexpr (kBig) {
    if (it.parts == 4) gemm_tile<kBf16, AL, BL, WI, 1, BK, RING, false>(g, t, smem, emit);
    else if (it.parts == 2) gemm_tile<kBf16, AL, BL, WI, 2, BK, RING, false>(g, t, smem, emit);
    else if (t.rows <= 64) gemm_tile<kBf16, AL, BL, 1, WJ, BK, RING, false>(g, t, smem, emit);
    else if (t.rows <= 128) gemm_tile<kBf16, AL, BL, 2, WJ, BK, RING, false>(g, t, smem, emit);
    else gemm_tile<kBf16, AL, BL, WI, WJ, BK, RING, false>(g, t, smem, emit);
  } else {
    gemm_tile<kBf16, AL, BL, WI, WJ, BK, RING, false>(g, t, smem, emit);
  }
}

}  // namespace mxt
