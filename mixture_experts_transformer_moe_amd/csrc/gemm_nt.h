// One tile of C = A B^T, both operands row-major with the reduction along the
// rows, bf16 with fp32 accumulation (v_mfma_f32_32x32x16_bf16).
//
// A workgroup of 4 waves (WR x WC) computes BM = 32 MB WR rows of A against
// BN = 32 NB WC rows of B.  B's operand comes first in the MFMA: in an
// accumulator lane l holds row l mod 32 of A's block, and its registers rows
// mfma32_row(r, l) of B's (four consecutive ones a quad).
//   * K advances in stages of 64 = one whole 128-byte line of each row, by direct
//     global->LDS loads into two buffers; the 16-byte pieces of row r are
//     XOR-swizzled by (r / 2) mod 8, conflict-free for the operand reads.
//   * One barrier a stage, before its last 16-wide MFMA step: by then every wave
//     has read the stage's last operands (a step ahead, into a second register
//     set), so the loads of the stage after the next go into its buffer, and the
//     next stage has landed: it was issued three steps before.
//   * Rows past the last are the last row again (their results are not stored).
//     K is a multiple of 8; pieces past its end read zeros.
//   * AT, BT: that operand lies the other way, [K, its rows] with the reduction from
//     row to row (its width a multiple of 8).  A stage is then 64 of its rows, 16-byte
//     units of row r XOR-swizzled by 4 (r mod 4), and gfx950's transposing LDS read
//     hands a lane 4 consecutive rows of one column, two reads an operand: in a group
//     of 16 lanes it returns to lane 4a + b element b of the 8-byte pieces addressed
//     by lanes a, a + 4, a + 8 and a + 12.  Rows past the reduction's end are its last
//     one again: the other operand has to hold zeros there.
#pragma once

#include <type_traits>
#include <utility>

#include "lds_dma.h"

namespace moe {

constexpr int kNtThreads = 256;
constexpr int kNtBK = 64;

// 16 bytes of zeros: the source of pieces past the reduction's end
__device__ const uint4 kNtZeros = {0u, 0u, 0u, 0u};

template <int WR_, int WC_, int MB_, int NB_>
struct NtShape {
  static constexpr int WR = WR_, WC = WC_, MB = MB_, NB = NB_;
  static constexpr int BM = 32 * MB * WR, BN = 32 * NB * WC;
  static constexpr int kStage = (BM + BN) * kNtBK * 2;       // bytes of a stage
  static constexpr int kLds = 2 * kStage;
  static_assert(WR * WC == 4 && BM % 32 == 0 && BN % 32 == 0, "four waves");
};

struct NtOperand {
  const bf16_t* p;     // the tile's first row (AT, BT: its first column in row 0)
  int ld;              // elements between rows, a multiple of 8
  int rows;            // rows from p on that exist (>= 1; AT, BT: columns, a multiple of 8)
  int depth;           // AT, BT: rows of the reduction that exist (>= 1)
};

typedef short nt_v4i16 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint2 nt_read_tr(uint32_t at) {
  typedef __attribute__((address_space(3))) nt_v4i16 lds_v4;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (lds_v4*)(reinterpret_cast<__attribute__((address_space(3))) bf16_t*>(at))));
}

// a lane's piece of a transposed stage with rows of `units` 16-byte units: row 8 (lane /
// 32) + (lane mod 16) / 4 of a step, by the operand's block of 32 columns
__device__ __forceinline__ uint32_t nt_tr_at(int lane, int block, int units) {
  const int tgrp = lane >> 4, tj = lane & 15;
  return static_cast<uint32_t>((8 * (tgrp >> 1) + (tj >> 2)) * (units * 16) +
                               (((4 * block + 2 * (tgrp & 1) + ((tj & 3) >> 1)) ^ (4 * (tj >> 2))) << 4) + 8 * (tj & 1));
}

// the operand of 16-wide step s of such a stage
__device__ __forceinline__ u32x4 nt_read_step(uint32_t at, int row_bytes, int s) {
  const uint2 lo = nt_read_tr(at + 16 * s * row_bytes), hi = nt_read_tr(at + (16 * s + 4) * row_bytes);
  return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// a pointer that is the same in every lane, made visibly so
template <typename T>
__device__ __forceinline__ const T* nt_uniform(const T* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v)));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32)));
  return reinterpret_cast<const T*>((static_cast<uint64_t>(hi) << 32) | lo);
}

template <int OFF>
__device__ __forceinline__ void nt_dma(const unsigned char* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(voff), "s"(base), "s"(lds), "i"(OFF)
               : "memory", "m0", "scc");
}

__device__ __forceinline__ int nt_swizzle(int r) { return (r >> 1) & 7; }

// s_waitcnt immediate that waits for lgkmcnt <= n only (gfx9 encoding)
constexpr int nt_lgkm_only(int n) { return 15 | (7 << 4) | ((n & 15) << 8) | (3 << 14); }

template <class F, int... Q>
__device__ __forceinline__ void nt_each(F&& f, std::integer_sequence<int, Q...>) {
  (f(std::integral_constant<int, Q>{}), ...);
}

// pre(): run once the first two stages' loads are under way
template <class S, bool AT = false, bool BT = false, class Pre>
__device__ __forceinline__ void gemm_nt(const NtOperand& a, const NtOperand& b, int K, unsigned char* smem,
                                        f32x16 (&acc)[S::MB][S::NB], Pre&& pre) {
  static_assert((!AT || S::BM >= 128) && (!BT || S::BN >= 128), "the swizzle of transposed rows takes 16 units");
  constexpr int MB = S::MB, NB = S::NB;
  constexpr int NA = S::BM / 32, NBL = S::BN / 32;           // 1 KB loads of a wave and stage
  constexpr int NQ = NA + NBL;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / S::WC, wc = wave % S::WC;
  const int nk = (K + kNtBK - 1) / kNtBK;
  const bool ragged = K % kNtBK != 0;

  // load q of a wave: rows 8 (NA wave + q) .. + 7 of A's tile, then the same of B's
  // (transposed: the stage's rows, 512 / BM or BN of them a load)
  auto units = [](bool of_a) { return (of_a ? S::BM : S::BN) / 8; };   // 16-byte units of a transposed row
  auto index = [&](int q) { return q < NA ? NA * wave + q : NBL * wave + q - NA; };
  auto tr_row = [&](int q) { return 64 / units(q < NA) * index(q) + lane / units(q < NA); };
  auto tr_col = [&](int q) {
    return min(8 * ((lane % units(q < NA)) ^ (4 * (tr_row(q) & 3))), (q < NA ? a.rows : b.rows) - 8);
  };
  auto offset = [&](int r, int c, int ld) {
    return (static_cast<uint32_t>(r) * static_cast<uint32_t>(ld) + static_cast<uint32_t>(c)) * 2u;
  };
  uint32_t off[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const bool of_a = q < NA;
    const int ld = of_a ? a.ld : b.ld;
    if (of_a ? AT : BT) {
      off[q] = offset(tr_row(q), tr_col(q), ld);
    } else {
      const int row = 8 * index(q) + (lane >> 3);
      off[q] = offset(min(row, (of_a ? a.rows : b.rows) - 1), 8 * ((lane & 7) ^ nt_swizzle(row)), ld);
    }
  }
  const unsigned char* pa = reinterpret_cast<const unsigned char*>(nt_uniform(a.p));
  const unsigned char* pb = reinterpret_cast<const unsigned char*>(nt_uniform(b.p));
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  // LDS: buffer s: A's rows, then B's
  auto issue = [&](int kb, int buf, auto q_tag, bool last) __attribute__((always_inline)) {
    constexpr int q = decltype(q_tag)::value;
    constexpr bool of_a = q < NA, tr = of_a ? AT : BT;
    const NtOperand& x = of_a ? a : b;
    const unsigned char* base = (of_a ? pa : pb) + kb * (tr ? static_cast<size_t>(x.ld) * (kNtBK * 2) : kNtBK * 2);
    const uint32_t at = lds0 + static_cast<uint32_t>(buf) * S::kStage +
                        (of_a ? NA * 1024u * wave : S::BM * 128u + NBL * 1024u * wave);
    constexpr int kAt = (of_a ? q : q - NA) * 1024;
    if (tr && last) {
      nt_dma<kAt>(base, offset(min(tr_row(q), x.depth - 1 - kb * kNtBK), tr_col(q), x.ld),
                  __builtin_amdgcn_readfirstlane(at));
    } else if (!tr && last && ragged) {
      // the last stage of a ragged reduction: pieces past its end are zeros
      const int row = 8 * index(q) + (lane >> 3);
      const int col = kb * kNtBK + 8 * ((lane & 7) ^ nt_swizzle(row));
      const void* from = col < K ? static_cast<const void*>(base + off[q]) : static_cast<const void*>(&kNtZeros);
      dma16(from, __builtin_amdgcn_readfirstlane(at + kAt));
    } else {
      nt_dma<kAt>(base, off[q], __builtin_amdgcn_readfirstlane(at));
    }
  };
  // the loads Q of a stage for which NM Q / NQ is k (all of them: k = -1)
  constexpr int NM = MB * NB, NR = MB + NB;                  // MFMAs and reads of a step
  auto issue_at = [&](int kb, int buf, int k, bool last) __attribute__((always_inline)) {
    nt_each([&](auto q) __attribute__((always_inline)) {
      if (k < 0 || NM * decltype(q)::value / NQ == k) issue(kb, buf, q, last);
    }, std::make_integer_sequence<int, NQ>{});
  };

  // operand reads: A block m of this wave is tile rows 32 (MB wr + m) .. + 31
  const int r32 = lane & 31;
  uint32_t piece_off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
    piece_off[s] = static_cast<uint32_t>(r32 * 128 + (((2 * s + (lane >> 5)) ^ nt_swizzle(r32)) << 4));
  struct Frag {
    u32x4 a[MB], b[NB];
  };
  uint32_t tr_a[MB], tr_b[NB];
#pragma unroll
  for (int m = 0; m < MB; ++m) tr_a[m] = AT ? nt_tr_at(lane, MB * wr + m, S::BM / 8) : 0u;
#pragma unroll
  for (int n = 0; n < NB; ++n) tr_b[n] = BT ? nt_tr_at(lane, NB * wc + n, S::BN / 8) : 0u;
  auto read_one = [&](Frag& f, int buf, int s, int i) __attribute__((always_inline)) {
    const unsigned char* base = smem + buf * S::kStage;
    const uint32_t at = lds0 + static_cast<uint32_t>(buf) * S::kStage;
    if (i < NB) {
      if constexpr (BT) f.b[i] = nt_read_step(at + S::BM * 128 + tr_b[i], S::BN * 2, s);
      else f.b[i] = *reinterpret_cast<const u32x4*>(base + S::BM * 128 + (NB * wc + i) * 4096 + piece_off[s]);
    } else {
      if constexpr (AT) f.a[i - NB] = nt_read_step(at + tr_a[i - NB], S::BM * 2, s);
      else f.a[i - NB] = *reinterpret_cast<const u32x4*>(base + (MB * wr + i - NB) * 4096 + piece_off[s]);
    }
  };
  auto mfma = [&](const Frag& f, auto&& op) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, f.b[n]),
                                                            __builtin_bit_cast(bf16x8, f.a[m]), acc[m][n], 0, 0, 0);
        op(m * NB + n);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  // the reads of the next step are spread over a step's MFMAs
  auto reads_at = [&](Frag& f, int buf, int s, int k) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (i * NM / NR == k) read_one(f, buf, s, i);
  };

#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x16{0.f};
  issue_at(0, 0, -1, nk == 1);
  if (nk > 1) issue_at(1, 1, -1, nk == 2);
  pre();                                                      // (its loads only add to what the wait leaves out)
  if (nk > 1) __builtin_amdgcn_s_waitcnt(vmcnt_only(NQ));
  else __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frag f0, f1;
#pragma unroll
  for (int i = 0; i < NR; ++i) read_one(f0, 0, 0, i);
  // stage kb; NEXT: what is issued for the stage after the next (0 nothing, 1 a
  // whole stage, 2 the last one)
  auto stage = [&](int kb, auto next_tag) __attribute__((always_inline)) {
    constexpr int NEXT = decltype(next_tag)::value;
    const int p = kb & 1;
    mfma(f0, [&](int k) __attribute__((always_inline)) { reads_at(f1, p, 1, k); });
    mfma(f1, [&](int k) __attribute__((always_inline)) { reads_at(f0, p, 2, k); });
    mfma(f0, [&](int k) __attribute__((always_inline)) { reads_at(f1, p, 3, k); });
    // this wave's reads of the stage are done, its loads of the next have landed
    __builtin_amdgcn_s_waitcnt(nt_lgkm_only(0));
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    mfma(f1, [&](int k) __attribute__((always_inline)) {
      reads_at(f0, p ^ 1, 0, k);                              // (after the last stage: not used)
      if constexpr (NEXT != 0) issue_at(kb + 2, p, k, NEXT == 2);
    });
  };
  int kb = 0;
  for (; kb + 3 < nk; ++kb) stage(kb, std::integral_constant<int, 1>{});
  if (kb + 2 < nk) stage(kb++, std::integral_constant<int, 2>{});
  for (; kb < nk; ++kb) stage(kb, std::integral_constant<int, 0>{});
  __syncthreads();                                            // the buffers are free
}

// Tile order for 8 XCDs (workgroup b runs on XCD b mod 8): each XCD takes a run of
// consecutive tiles, and consecutive tiles are blocks of 4 row tiles of A by the
// column tiles, so that the 32 tiles that run on an XCD at a time share 4 panels
// of A and 8 of B behind one L2.  Where a reduction comes in parts the run goes
// through the tiles of part z, then of the next: they share the part's panels (dx of 333
// rows x 1000 in 21 parts of 33001: 30 us, 48 with a part's 24 tiles spread over the XCDs).
__device__ __forceinline__ void nt_tile(int b, int tiles_m, int tiles_n, int parts, int& tm, int& tn, int& z) {
  const int tiles = tiles_m * tiles_n, n = tiles * parts;
  const int x = b % 8, i = b / 8, q = n / 8, rem = n % 8;
  int t = x * q + min(x, rem) + i;
  z = t / tiles;
  t -= z * tiles;
  const int group = t / (4 * tiles_n), m0 = 4 * group;
  const int gm = min(4, tiles_m - m0), in = t - group * 4 * tiles_n;
  tm = m0 + in % gm;
  tn = in / gm;
}

}  // namespace moe
