// Experts' products with 4-bit weights and group scales, bf16 activations, fp32
// accumulation; the quantisation of bf16 weights and the packing of given codes.
//
// What they compute ("Laguna M.1/XS.2 Technical Report", Key claims: INT4
// quantised MoE layers; "Laguna-M.1-base", Feed-forward: SwiGLU without biases):
// with q[r, c] in -8..7 and one bf16 scale s[r, c / G] a row and group of G columns,
//   y[p, r] = sum_g s[r, g] sum_{c in g} q[r, c] a[p, c]
//   gate_up  h[p] = silu(y_gate) * y_up;   down  y[p]
// for the rows p of each expert, and for the shared expert over all tokens.
//
// Numbers.  A code is stored as q + 8 and widened to q in bf16, exactly (widen), so
// that products are exact and sums are fp32 sums of the terms themselves: a code of 0
// adds nothing, whatever its activation.  (128 + code would be one AND-OR for two
// codes, but its offset has to leave again through the sum and leaves a rounding of
// 136 sum |a|: 5e-4 instead of 0 for weights of zero under unit activations with
// outliers of 50, and a fifth more MFMAs.  Exact codes cost decode 4%, 32 tokens at the
// M.1 widths 67 -> 69 us, and one token 12.7 -> 14.8 us; long prompts gain 5%.)  A group's
// sum is then multiplied by its scale in fp32.
//
// Layout.  Blocks of 16 rows x 128 columns, 1 KB, row-block major: lane l's 16
// bytes are its codes of four 16x16x32 MFMA steps, row l mod 16, columns
// 32 i + 8 (l / 16) .. + 7 of dword i, element e in nibble e / 2 + 4 (e mod 2).
#include "int4.h"

#include <type_traits>

#include "grouped_gemm.h"
#include "int4_plan.h"
#include "mma_stream.h"

namespace moe {
namespace {

enum Int4Mode { kInt4GateUp = 0, kInt4Down = 1 };

constexpr int kRowBlock = 16;          // weight rows of a packed block
constexpr int kColBlock = 128;         // its columns
constexpr int kBlockBytes = 1024;

struct Int4Args {
  const bf16_t* a_routed;    // [S, K] rows in expert order, or x when gather != null
  const int32_t* gather;     // sorted_token, or null
  const bf16_t* a_shared;    // [T, Ks]
  const uint8_t* w_routed;   // E packed [Nw, K] matrices
  const uint8_t* w_shared;
  const bf16_t* s_routed;    // [E, Nw, K / G]
  const bf16_t* s_shared;    // [Nws, Ks / G]
  bf16_t* out_routed;        // [S, N]
  bf16_t* out_shared;        // [T, Ns]
  const int32_t* offsets;    // [E + 1]
  int T, E, S;
  int K, Ks, N, Ns;
  int tiles_r, tiles_s;      // column tiles of a routed expert, of the shared one
  int ks_r, ks_s;            // waves of a workgroup that share a tile's reduction
};

// Eight codes q + 8 -> q in bf16.  gfx950 converts two E4M3 bytes at a time, and a byte up
// to 15 counts 2^-9 there (8 and up are the lowest normal binade): so magnitudes and signs
// of all eight in their nibbles first, then in bytes, the even nibbles' and the odd ones'.
// Those are elements 0 4 1 5 and 2 6 3 7; unless IN_ORDER the operand keeps that order, and
// the activations take it too (reorder).  12 instructions, 14 in order.
template <bool IN_ORDER>
__device__ __forceinline__ bf16x8 widen(uint32_t w) {
  // (as three-operand logic: written out, the compiler makes more of it)
  auto and_not = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_bitop3_b32(a, b, b, 0x30); };   // a & ~b
  auto choose = [](uint32_t a, uint32_t m, uint32_t b) { return __builtin_amdgcn_bitop3_b32(a, m, b, 0xe2); };   // m ? a : b
  const uint32_t low = 0x0f0f0f0fu;
  const uint32_t minus = and_not(0x88888888u, w), one = minus >> 3;
  const uint32_t mag = (w ^ (0x88888888u - one)) + one;    // code below 8: 7 - code + 1; else code - 8
  uint32_t even = choose(mag, low, minus << 4), odd = choose(mag >> 4, low, minus);
  if constexpr (IN_ORDER) {
    even = __builtin_amdgcn_perm(even, even, 0x03010200u);
    odd = __builtin_amdgcn_perm(odd, odd, 0x03010200u);
  }
  auto pair = [](uint32_t v, auto high) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.0f, decltype(high)::value));
  };
  const std::false_type lo{};
  const std::true_type hi{};
  // in order: elements 0 1 4 5 | 2 3 6 7
  const u32x4 v = IN_ORDER ? u32x4{pair(even, lo), pair(odd, lo), pair(even, hi), pair(odd, hi)}
                           : u32x4{pair(even, lo), pair(even, hi), pair(odd, lo), pair(odd, hi)};
  return __builtin_bit_cast(bf16x8, v);
}

// eight activations in the order of widen<false>'s elements
__device__ __forceinline__ u32x4 reorder(const u32x4& x) {
  auto lows = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); };
  auto highs = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); };
  return u32x4{lows(x[0], x[2]), highs(x[0], x[2]), lows(x[1], x[3]), highs(x[1], x[3])};
}

// 16 bytes at a base that is the same in every lane plus the lane's own offset.
// The offset is made opaque where it is used: otherwise the compiler adds the two
// outside the loop and holds a 64-bit address for every load.
template <bool NT>
__device__ __forceinline__ u32x4 load16(const void* base, uint32_t off) {
  asm volatile("" : "+v"(off));
  const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const unsigned char*>(base) + off);
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}

// Between LDS writes of some of a wave's lanes and reads of others, both ways: the
// hardware does a wave's LDS operations in order, and the compiler, which sees one lane
// at a time, moves none across.  No instruction.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// One workgroup: a column tile of one expert, its rows up to 16 TM at a time.  Four
// waves of 64 weight rows each (gate_up: 32 gate rows and the up rows of the same
// columns): ks of them share the reduction, 4 / ks stand side by side.  Weights go
// straight into registers, a block ahead; rows and scales are read as whole lines
// and turned into operands through the wave's own LDS (read as operands they are
// 16- and 2-byte pieces of many lines: 87 us against 75 for 32 tokens' gate/up at
// D = 4096, F = 1024).  No barrier before the waves' parts meet.
template <int MODE, int TM, int G>
__global__ __launch_bounds__(256, TM == 1 ? 3 : 2) void int4_rows_kernel(Int4Args a) {
  constexpr int NB = 4;                                   // 16-row weight blocks of a wave
  constexpr int kCols = MODE == kInt4GateUp ? 32 : 64;    // output columns of a wave
  constexpr int GC = kColBlock / G;                       // groups of a packed block
  constexpr int kAhead = TM == 2 ? 4 : 2;                 // blocks of weights in flight (TM 1: 2 and 3 workgroups a CU
                                                          // beat 4 and 2 by 5% to 25%)
  constexpr int kRun = 8;                                 // blocks whose scales are in LDS at a time
  constexpr int NG = kRun * GC;                           // groups of a run
  constexpr int kScaleLd = NG + 2;                        // (an odd number of words: no bank conflicts)
  constexpr int kRowsBytes = 16 * TM * 2 * kColBlock;     // a block's columns of the rows
  constexpr int kWaveBytes = kRowsBytes + 64 * kScaleLd * 2;
  constexpr int kPartBytes = 4 * NB * TM * 256 * 4;
  __shared__ __attribute__((aligned(16))) unsigned char
      smem[4 * kWaveBytes > kPartBytes ? 4 * kWaveBytes : kPartBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // ---- whose tile: chunk by chunk the shared expert's rows first, then each
  // expert's.  Lane l counts the chunks of experts 4 l .. 4 l + 3.
  constexpr int kChunk = 16 * TM;
  int bid = blockIdx.x;
  const int chunks_s = a.tiles_s > 0 ? (a.T + kChunk - 1) / kChunk : 0;
  const bool shared = bid < a.tiles_s * chunks_s;
  int e = 0, lo = 0, M = a.T, tile, m0;
  if (shared) {
    m0 = bid / a.tiles_s * kChunk;
    tile = bid % a.tiles_s;
  } else {
    bid -= a.tiles_s * chunks_s;
    const int slot = bid / a.tiles_r;
    tile = bid % a.tiles_r;
    static_assert(kGemmMaxE == 4 * 64, "four experts a lane");
    int off[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) off[j] = a.offsets[min(4 * lane + j, a.E)];
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      // clamped so that no offsets table can move a row outside [0, S)
      off[j] = min(max(off[j], j ? off[j - 1] : 0), a.S);
      if (j) sum += (off[j] - off[j - 1] + kChunk - 1) / kChunk;
    }
    int end = sum;                                        // inclusive scan
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(end, d);
      if (lane >= d) end += v;
    }
    const uint64_t here = __ballot(slot < end);           // the first lane past the slot
    if (here == 0) return;
    const int src = __ffsll(static_cast<unsigned long long>(here)) - 1;
    int left = slot - (end - sum), j = 0;                 // (of use in lane src)
#pragma unroll
    for (int q = 1; q < 4; ++q) {
      const int n = (off[q] - off[q - 1] + kChunk - 1) / kChunk;
      if (j == q - 1 && left >= n) {
        left -= n;
        j = q;
      }
    }
    const int from = j == 0 ? off[0] : (j == 1 ? off[1] : (j == 2 ? off[2] : off[3]));
    const int to = j == 0 ? off[1] : (j == 1 ? off[2] : (j == 2 ? off[3] : off[4]));
    e = min(__builtin_amdgcn_readlane(4 * lane + j, src), a.E - 1);
    lo = __builtin_amdgcn_readlane(from, src);
    M = __builtin_amdgcn_readlane(to, src) - lo;
    m0 = __builtin_amdgcn_readlane(left, src) * kChunk;
  }
  const int K = shared ? a.Ks : a.K;
  const int N = shared ? a.Ns : a.N;
  const int ks = shared ? a.ks_s : a.ks_r;
  const int rs = 4 / ks;
  const int Nw = MODE == kInt4GateUp ? 2 * N : N;
  const int ncb = K / kColBlock;                          // (even: K is a multiple of 256)
  const int kpart = wave % ks, side = wave / ks;
  const int c0 = 2 * (ncb / 2 * kpart / ks), c1 = 2 * (ncb / 2 * (kpart + 1) / ks);
  const int n0 = (tile * rs + side) * kCols;

  // ---- weights and scales of the wave's four blocks
  const uint8_t* wmat = shared ? a.w_shared : a.w_routed + static_cast<size_t>(e) * Nw * (K / 2);
  const bf16_t* smat = shared ? a.s_shared : a.s_routed + static_cast<size_t>(e) * Nw * (K / G);
  auto first_row = [&](int b) {                           // of weight block b
    return MODE == kInt4GateUp ? (b < 2 ? n0 + 16 * b : N + n0 + 16 * (b - 2)) : n0 + 16 * b;
  };
  const uint8_t* wb[NB];                                  // (the same in every lane)
  const bf16_t* sb[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    wb[b] = wmat + static_cast<size_t>(first_row(b) / kRowBlock) * ncb * kBlockBytes;
    sb[b] = smat + static_cast<size_t>(first_row(b)) * (K / G);
  }
  unsigned char* my_rows = smem + wave * kWaveBytes;
  uint32_t* my_scales = reinterpret_cast<uint32_t*>(my_rows + kRowsBytes);

  // the scales of the wave's 64 rows and a run of 8 blocks, two groups a word: word
  // i of a run holds groups 2 (i mod kP) .. + 1 of row i / kP
  constexpr int kP = NG / 2;
  struct Run {
    uint32_t v[kP];
  };
  auto load_run = [&](Run& r, int cs) __attribute__((always_inline)) {
    int ln = lane;
    asm volatile("" : "+v"(ln));                          // (the addresses are not kept in registers)
    const int word = min(ln % kP, (c1 - cs) * GC / 2 - 1);  // inside the wave's part
    const uint32_t off = (static_cast<uint32_t>(ln / kP) * static_cast<uint32_t>(K / G) + 2u * word) * 2u;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      constexpr int kRows = 64 / kP;                      // rows of a load
      const bf16_t* from = sb[j * kRows / 16] + (j * kRows % 16) * (K / G) + cs * GC;
      r.v[j] = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const unsigned char*>(from) + off);
    }
  };
  auto keep_run = [&](const Run& r) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kP; ++j) my_scales[(j * (64 / kP) + lane / kP) * (kScaleLd / 2) + lane % kP] = r.v[j];
  };

  // rows m0 .. m0 + 4 NI - 1
  auto chunk = [&](auto ni_tag) __attribute__((always_inline)) {
    constexpr int NI = decltype(ni_tag)::value;
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));      // per-lane arithmetic stays inside its variant
    constexpr int TB = (NI + 3) / 4;                      // token blocks of 16
    u32x4 ring[kAhead][NB];                               // weights of the next blocks
    u32x4 rows[NI];                                       // the next block's, on their way to LDS
    // load i: row 4 i + lane / 16, its 16-byte piece lane mod 16 of a block's 256
    // bytes; in LDS piece c of row r sits at slot c ^ (r mod 16) (no bank conflicts
    // either way)
    const bf16_t* base = shared ? a.a_shared + static_cast<size_t>(m0) * K
                                : (a.gather ? a.a_routed : a.a_routed + static_cast<size_t>(lo + m0) * K);
    uint32_t xo[NI];
    int tok[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = min(4 * i + (lane >> 4), M - 1 - m0);
      tok[i] = !shared && a.gather ? a.gather[lo + m0 + row] : row;
    }
    f32x4 acc[TB][NB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto load = [&](u32x4 (&w)[NB], int cb) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        w[b] = load16<true>(wb[b] + static_cast<size_t>(cb < c1 ? cb : c0) * kBlockBytes, cb < c1 ? lane * 16u : 0u);
    };
    auto load_rows = [&](int cb) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) rows[i] = load16<false>(base + (cb < c1 ? cb : c0) * kColBlock, cb < c1 ? xo[i] : 0u);
    };
    auto keep_rows = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = 4 * i + (lane >> 4);
        *reinterpret_cast<u32x4*>(my_rows + r * 256 + (((lane & 15) ^ (r & 15)) << 4)) = reorder(rows[i]);
      }
    };
    auto compute = [&](const u32x4 (&wq)[NB], int j, bool odd) __attribute__((always_inline)) {   // block j of the run
      constexpr int SG = 4 / GC;                         // MFMA steps of a group
      // (tokens past 4 NI - 1 hold what was there, and only outputs that are not
      // stored depend on them)
      bf16x8 x[TB][4];
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[t][i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
                                                   my_rows + (16 * t + (lane & 15)) * 256 +
                                                   (((4 * i + (lane >> 4)) ^ (lane & 15)) << 4)));
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        // the scale of row `lane` of the wave's 64, then those of rows lane mod 16
        // of each block
        const uint32_t two = my_scales[lane * (kScaleLd / 2) + (j * GC + g) / 2];
        const uint32_t own = (GC == 1 ? odd : g % 2 != 0) ? two & 0xffff0000u : two << 16;
        const auto p = __builtin_amdgcn_permlane32_swap(own, own, false, false);       // rows 0 1 0 1, 2 3 2 3
        const auto p01 = __builtin_amdgcn_permlane16_swap(p[0], p[0], false, false);
        const auto p23 = __builtin_amdgcn_permlane16_swap(p[1], p[1], false, false);
        const float sc[NB] = {__uint_as_float(p01[0]), __uint_as_float(p01[1]), __uint_as_float(p23[0]),
                              __uint_as_float(p23[1])};
        // a step of all blocks at a time: NB TB chains side by side
        f32x4 y[TB][NB];
#pragma unroll
        for (int i = 0; i < SG; ++i) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const bf16x8 w = widen<false>(wq[b][g * SG + i]);
#pragma unroll
            for (int t = 0; t < TB; ++t)
              y[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t][g * SG + i], w, i == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : y[t][b],
                                                                0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);              // a step's operands at a time
        }
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][b][r] = fmaf(sc[b], y[t][b][r], acc[t][b][r]);
      }
    };
    // kAhead blocks of weights in flight; the loads are unconditional (past the end
    // every lane reads the same 16 bytes), so that the waits before a block leave
    // those of the later ones in flight
    if (c0 < c1) {
      Run run;
      load_run(run, c0);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) load(ring[q], c0 + q);
      __builtin_amdgcn_sched_barrier(0);                  // the weights are under way before the rows' ids are here
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int row = !shared && a.gather ? min(max(tok[i], 0), a.T - 1) : tok[i];
        xo[i] = (static_cast<uint32_t>(row) * static_cast<uint32_t>(K) + 8u * (lane & 15)) * 2u;
      }
      load_rows(c0);
      for (int cb = c0; cb < c1; cb += kAhead) {
        if ((cb - c0) % kRun == 0) {
          keep_run(run);
          load_run(run, min(cb + kRun, c1 - 2));
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          keep_rows();
          wave_lds_fence();
          load_rows(cb + q + 1);
          if (cb + q < c1) compute(ring[q], (cb - c0) % kRun + q, q % 2 != 0);
          wave_lds_fence();
          load(ring[q], cb + q + kAhead);
        }
      }
    }

    // ---- the waves' parts meet in LDS: [wave][tb][block][token][row]
    float* part = reinterpret_cast<float*>(smem);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          part[((wave * TB + t) * NB + b) * 256 + (4 * (lane >> 4) + r) * 16 + (lane & 15)] = acc[t][b][r];
    __syncthreads();
    constexpr int kPairs = kCols / 2;                     // column pairs of a side
    const int left = min(M - m0, 4 * NI);
    for (int i = tid; i < rs * left * kPairs; i += 256) {
      const int c = 2 * (i % kPairs), rest = i / kPairs;
      const int m = rest % left, sd = rest / left;
      auto sum = [&](int b, int r) {
        float v = 0.f;
        for (int k = 0; k < ks; ++k)
          v += part[(((sd * ks + k) * TB + m / 16) * NB + b) * 256 + (m % 16) * 16 + r];
        return v;
      };
      float y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = (c + j) / 16, r = (c + j) % 16;
        y[j] = sum(b, r);
        if constexpr (MODE == kInt4GateUp) {
          const float up = sum(b + 2, r);
          y[j] = y[j] * __builtin_amdgcn_rcpf(1.0f + __expf(-y[j])) * up;
        }
      }
      bf16_t* out = shared ? a.out_shared : a.out_routed + static_cast<size_t>(lo) * N;
      *reinterpret_cast<uint32_t*>(out + static_cast<size_t>(m0 + m) * N + (tile * rs + sd) * kCols + c) =
          pack_bf16x2(y[0], y[1]);
    }
  };
  // with as few row loads as hold the chunk
  const int left = M - m0;
  if (TM > 1 && left > 16) chunk(std::integral_constant<int, 4 * TM>{});
  else if (left > 4) chunk(std::integral_constant<int, 4>{});
  else chunk(std::integral_constant<int, 1>{});
}

// Many rows an expert: one workgroup computes 128 rows x 256 weight rows (gate_up:
// 128 gate rows and the up rows of the same columns) over the whole reduction, a
// wave 64 of the weight rows (as above) and all 128 rows.  The rows' columns come
// 128 at a time by direct global->LDS loads into two buffers, whole lines, the
// 16-byte pieces of row r XOR-swizzled by r mod 16; weights go straight into
// registers half a stage ahead and are widened once for the 8 token blocks.  At most
// 64 columns are summed before the scales: 32 operand registers a wave, so that two
// workgroups share a CU and one's conversions run beside the other's MFMAs.
// Tiles in order of expert, column tile, row block, each XCD a run of them, so that
// an expert's rows and a column tile's weights stay behind one L2.  An expert's rows
// are split evenly, and each number of token blocks has its own loop: 4096 tokens at
// D = 4096, F = 1024 (128 rows an expert) gate/up 705 us, 755 with blocks of 128 rows and
// a rest and every second number, 778 split evenly with every second number; down 396, 418
// and 407.
template <int MODE, int G>
__global__ __launch_bounds__(256, 2) void int4_tile_kernel(Int4Args a) {
  constexpr int NB = 4, TB = 8, kRows = 16 * TB;
  constexpr int kCols = MODE == kInt4GateUp ? 32 : 64;    // output columns of a wave
  constexpr int GC = kColBlock / G;                       // scales of a row and block
  constexpr int kStage = kRows * kColBlock * 2;           // 32 KB
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // ---- whose tile (the shared expert's first); lane l counts experts 4 l .. 4 l + 3
  const int chunks_s = a.tiles_s > 0 ? (a.T + kRows - 1) / kRows : 0;
  int off[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) off[j] = a.offsets[min(4 * lane + j, a.E)];
  int sum = 0;
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    off[j] = min(max(off[j], j ? off[j - 1] : 0), a.S);
    if (j) sum += (off[j] - off[j - 1] + kRows - 1) / kRows;
  }
  int end = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(end, d);
    if (lane >= d) end += v;
  }
  const int n_s = chunks_s * a.tiles_s;
  const int total = n_s + __builtin_amdgcn_readlane(end, 63) * a.tiles_r;
  const int xcd = blockIdx.x % kGemmXcds, in_xcd = blockIdx.x / kGemmXcds;
  const int share = total / kGemmXcds, rem = total % kGemmXcds;
  if (in_xcd >= share + (xcd < rem ? 1 : 0)) return;
  int t = xcd * share + min(xcd, rem) + in_xcd;
  const bool shared = t < n_s;
  int e = 0, lo = 0, M = a.T, tile, chunk, chunks = chunks_s;
  if (shared) {
    chunk = t % chunks_s;
    tile = t / chunks_s;
  } else {
    t -= n_s;
    const int slot = t / a.tiles_r;
    const int src = __ffsll(static_cast<unsigned long long>(__ballot(slot < end))) - 1;
    int first = end - sum, j = 0;                         // chunks before expert 4 l + j
#pragma unroll
    for (int q = 1; q < 4; ++q) {
      const int n = (off[q] - off[q - 1] + kRows - 1) / kRows;
      if (j == q - 1 && slot >= first + n) {
        first += n;
        j = q;
      }
    }
    const int from = j == 0 ? off[0] : (j == 1 ? off[1] : (j == 2 ? off[2] : off[3]));
    const int to = j == 0 ? off[1] : (j == 1 ? off[2] : (j == 2 ? off[3] : off[4]));
    e = min(__builtin_amdgcn_readlane(4 * lane + j, src), a.E - 1);
    lo = __builtin_amdgcn_readlane(from, src);
    M = __builtin_amdgcn_readlane(to, src) - lo;
    const int local = t - __builtin_amdgcn_readlane(first, src) * a.tiles_r;
    chunks = (M + kRows - 1) / kRows;
    chunk = local % chunks;
    tile = local / chunks;
  }
  // as even row blocks as whole token blocks allow (none is empty: M > 128 (chunks - 1))
  const int size = (M + 16 * chunks - 1) / (16 * chunks) * 16, m0 = chunk * size;
  const int K = shared ? a.Ks : a.K;
  const int N = shared ? a.Ns : a.N;
  const int Nw = MODE == kInt4GateUp ? 2 * N : N;
  const int ncb = K / kColBlock;
  const int n0 = (tile * 4 + wave) * kCols;
  const int valid = min(size, M - m0);
  const int tbv = (valid + 15) / 16;                      // token blocks with rows

  // ---- sources
  const uint8_t* wmat = shared ? a.w_shared : a.w_routed + static_cast<size_t>(e) * Nw * (K / 2);
  const bf16_t* smat = shared ? a.s_shared : a.s_routed + static_cast<size_t>(e) * Nw * (K / G);
  auto first_row = [&](int b) {
    return MODE == kInt4GateUp ? (b < 2 ? n0 + 16 * b : N + n0 + 16 * (b - 2)) : n0 + 16 * b;
  };
  const uint8_t* wb[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) wb[b] = wmat + static_cast<size_t>(first_row(b) / kRowBlock) * ncb * kBlockBytes;
  // lane l loads the scales of row l of the wave's 64
  const bf16_t* sp = smat + static_cast<size_t>(first_row(lane >> 4) + (lane & 15)) * (K / G);
  // load q of a wave: rows 4 (8 wave + q) + lane / 16, slot lane mod 16
  const unsigned char* xbase = reinterpret_cast<const unsigned char*>(
      shared ? a.a_shared + static_cast<size_t>(m0) * K
             : (a.gather ? a.a_routed : a.a_routed + static_cast<size_t>(lo + m0) * K));
  uint32_t xo[TB];
#pragma unroll
  for (int q = 0; q < TB; ++q) {
    const int r = 4 * (TB * wave + q) + (lane >> 4);
    int row = min(r, valid - 1);
    if (!shared && a.gather) row = min(max(a.gather[lo + m0 + row], 0), a.T - 1);
    xo[q] = (static_cast<uint32_t>(row) * static_cast<uint32_t>(K) + 8u * ((lane & 15) ^ (r & 15))) * 2u;
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  auto issue_rows = [&](int cb) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < TB; ++q)
      dma16_off(xbase + static_cast<size_t>(cb) * (kColBlock * 2), xo[q],
                lds0 + static_cast<uint32_t>(cb & 1) * kStage + (TB * wave + q) * 1024u);
  };
  struct Stage {
    u32x4 w[NB];
    uint32_t s[(GC + 1) / 2];                             // GC scales, two a word (GC 1: one)
  };
  auto load = [&](Stage& f, int cb) __attribute__((always_inline)) {
    const bool in = cb < ncb;                             // (past the end every lane reads the same)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      f.w[b] = load16<false>(wb[b] + static_cast<size_t>(in ? cb : 0) * kBlockBytes, in ? lane * 16u : 0u);
    const bf16_t* from = sp + (in ? cb : 0) * GC;
    if constexpr (GC == 1) {
      f.s[0] = *from;
    } else {
#pragma unroll
      for (int g = 0; g < GC / 2; ++g) f.s[g] = reinterpret_cast<const uint32_t*>(from)[g];
    }
  };
  f32x4 acc[TB][NB];
#pragma unroll
  for (int i = 0; i < TB; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a stage over the row block's NT live token blocks
  auto compute = [&](Stage& f, int cb, auto nt_tag) __attribute__((always_inline)) {
    constexpr int NT = decltype(nt_tag)::value;
    const unsigned char* X = smem + (cb & 1) * kStage;
    constexpr int SG = G == 32 ? 1 : 2;                   // MFMA steps before the scales
#pragma unroll
    for (int part = 0; part < 4 / SG; ++part) {
      const int g = part * SG * 32 / G;                   // the group
      const uint32_t word = f.s[g / 2];
      const uint32_t own = GC == 1 || g % 2 == 0 ? word << 16 : word & 0xffff0000u;
      const auto p = __builtin_amdgcn_permlane32_swap(own, own, false, false);
      const auto p01 = __builtin_amdgcn_permlane16_swap(p[0], p[0], false, false);
      const auto p23 = __builtin_amdgcn_permlane16_swap(p[1], p[1], false, false);
      const float sc[NB] = {__uint_as_float(p01[0]), __uint_as_float(p01[1]), __uint_as_float(p23[0]),
                            __uint_as_float(p23[1])};
      bf16x8 w[SG][NB];
#pragma unroll
      for (int i = 0; i < SG; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) w[i][b] = widen<true>(f.w[b][part * SG + i]);
      // (the registers of the packed weights are free: the next stage's)
      if (part == 4 / SG - 1) load(f, cb + 1);
      auto read = [&](bf16x8 (&x)[SG], int i) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < SG; ++k)
          x[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
                                                X + (16 * i + (lane & 15)) * 256 +
                                                (((4 * (part * SG + k) + (lane >> 4)) ^ (lane & 15)) << 4)));
      };
      bf16x8 x[2][SG];
      read(x[0], 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (i + 1 < NT) read(x[(i + 1) & 1], i + 1);
        f32x4 y[NB];
#pragma unroll
        for (int k = 0; k < SG; ++k)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            y[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i & 1][k], w[k][b], k == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : y[b], 0, 0, 0);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][b][r] = fmaf(sc[b], y[b][r], acc[i][b][r]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // stage cb: its rows were issued a stage before, its weights half a stage
  Stage f;
  issue_rows(0);
  load(f, 0);
  auto k_loop = [&](auto nt_tag) __attribute__((always_inline)) {
    for (int cb = 0; cb < ncb; ++cb) {
      __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (cb + 1 < ncb) issue_rows(cb + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(f, cb, nt_tag);
    }
  };
  if (tbv > 7) k_loop(std::integral_constant<int, 8>{});
  else if (tbv > 6) k_loop(std::integral_constant<int, 7>{});
  else if (tbv > 5) k_loop(std::integral_constant<int, 6>{});
  else if (tbv > 4) k_loop(std::integral_constant<int, 5>{});
  else if (tbv > 3) k_loop(std::integral_constant<int, 4>{});
  else if (tbv > 2) k_loop(std::integral_constant<int, 3>{});
  else k_loop(std::integral_constant<int, 2>{});

  // ---- out through LDS: [row][the tile's columns], pieces of 16 bytes swizzled
  constexpr int kTileCols = 4 * kCols, kPieces = kTileCols / 8;
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
  __syncthreads();
  auto piece_at = [&](int row, int piece) { return smem + row * (kTileCols * 2) + ((piece ^ (((row >> 2) & 3) << 1)) << 4); };
#pragma unroll
  for (int i = 0; i < TB; ++i)
#pragma unroll
    for (int b = 0; b < kCols / 16; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[i][b][r];
        if constexpr (MODE == kInt4GateUp) v = v * __builtin_amdgcn_rcpf(1.0f + __expf(-v)) * acc[i][(b + 2) % NB][r];
        const int row = 16 * i + 4 * (lane >> 4) + r, col = kCols * wave + 16 * b + (lane & 15);
        *reinterpret_cast<bf16_t*>(piece_at(row, col >> 3) + 2 * (col & 7)) = f32_to_bf16(v);
      }
  __syncthreads();
  bf16_t* out = (shared ? a.out_shared : a.out_routed + static_cast<size_t>(lo) * N) + static_cast<size_t>(m0) * N + tile * kTileCols;
  for (int i = tid; i < valid * kPieces; i += 256) {
    const int row = i / kPieces, piece = i % kPieces;
    *reinterpret_cast<u32x4*>(out + static_cast<size_t>(row) * N + 8 * piece) =
        *reinterpret_cast<const u32x4*>(piece_at(row, piece));
  }
}

// ------------------------------------------------------------------ load time

// byte of the packed matrix that holds columns 8j .. 8j + 7 of row r as one dword
__device__ __forceinline__ int64_t int4_offset(int r, int c, int cols) {
  return (static_cast<int64_t>(r / kRowBlock) * (cols / kColBlock) + c / kColBlock) * kBlockBytes +
         ((r % kRowBlock) + 16 * ((c % 32) / 8)) * 16 + ((c % kColBlock) / 32) * 4;
}

// eight codes (4 bits each, element e in bits 4e) -> the packed dword
__device__ __forceinline__ uint32_t spread(uint32_t v) {
  uint32_t d = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) d |= ((v >> (4 * e)) & 15u) << (4 * (e / 2 + 4 * (e % 2)));
  return d;
}

__global__ __launch_bounds__(256) void pack_int4_kernel(const uint32_t* __restrict__ codes, uint8_t* __restrict__ dst,
                                                        int64_t count, int rows, int cols) {
  const int64_t per_mat = static_cast<int64_t>(rows) * cols / 8, all = count * per_mat;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t mi = i / per_mat, in = i - mi * per_mat;
    const int r = static_cast<int>(in / (cols / 8)), c = static_cast<int>(in % (cols / 8)) * 8;
    *reinterpret_cast<uint32_t*>(dst + mi * per_mat * 4 + int4_offset(r, c, cols)) = spread(codes[i]);
  }
}

// G / 8 threads a group: amax, scale = bf16(amax / 7) (1 where that is zero), codes
// of w / scale in fp32, ties to even
template <int G>
__global__ __launch_bounds__(256) void quantize_int4_kernel(const bf16_t* __restrict__ src, uint8_t* __restrict__ dst,
                                                            bf16_t* __restrict__ scales, int64_t nrows, int rows,
                                                            int cols) {
  constexpr int kT = G / 8;
  const int64_t units = nrows * (cols / 8);
  // (a group's threads sit in one wave and leave the loop together)
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < units;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t gr = i / (cols / 8);
    const int c = static_cast<int>(i % (cols / 8)) * 8;
    const uint4 v = *reinterpret_cast<const uint4*>(src + i * 8);
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
    float w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[2 * j] = __uint_as_float(d[j] << 16);
      w[2 * j + 1] = __uint_as_float(d[j] & 0xffff0000u);
    }
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(w[e]));
#pragma unroll
    for (int o = kT / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    bf16_t sb = f32_to_bf16(amax / 7.0f);
    if (sb == 0) sb = 0x3f80;
    const float s = bf16_to_f32(sb);
    uint32_t q = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = fminf(fmaxf(__builtin_rintf(w[e] / s), -8.0f), 7.0f);
      q |= (static_cast<uint32_t>(static_cast<int>(r) + 8) & 15u) << (4 * e);
    }
    const int64_t mi = gr / rows;
    *reinterpret_cast<uint32_t*>(dst + mi * rows * static_cast<int64_t>(cols / 2) +
                                 int4_offset(static_cast<int>(gr - mi * rows), c, cols)) = spread(q);
    if (c % G == 0) scales[gr * (cols / G) + c / G] = sb;
  }
}

template <int MODE, int TM>
hipError_t launch_rows(Int4Args a, int group, hipStream_t st) {
  constexpr int kCols = MODE == kInt4GateUp ? 32 : 64, kChunk = 16 * TM;
  // chunks the experts' rows can make
  const int64_t most = static_cast<int64_t>(a.E) + a.S / kChunk;
  const int64_t slots = a.S < most ? a.S : most;
  a.ks_r = int4_split(a.K / kColBlock, a.N, kCols, slots);
  a.tiles_r = a.N / (kCols * (4 / a.ks_r));
  const int64_t chunks_s = (a.T + kChunk - 1) / kChunk;
  a.ks_s = a.Ns > 0 ? int4_split(a.Ks / kColBlock, a.Ns, kCols, chunks_s) : 1;
  a.tiles_s = a.Ns > 0 ? a.Ns / (kCols * (4 / a.ks_s)) : 0;
  const int64_t grid = a.tiles_s * chunks_s + slots * a.tiles_r;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  switch (group) {
    case 32: int4_rows_kernel<MODE, TM, 32><<<static_cast<unsigned>(grid), 256, 0, st>>>(a); break;
    case 64: int4_rows_kernel<MODE, TM, 64><<<static_cast<unsigned>(grid), 256, 0, st>>>(a); break;
    default: int4_rows_kernel<MODE, TM, 128><<<static_cast<unsigned>(grid), 256, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_tiles4(Int4Args a, int group, hipStream_t st) {
  constexpr int kRows = 128, kTileCols = MODE == kInt4GateUp ? 128 : 256;
  a.tiles_r = a.N / kTileCols;
  a.tiles_s = a.Ns / kTileCols;
  const int64_t most = static_cast<int64_t>(a.E) + a.S / kRows;
  const int64_t tiles = (a.S < most ? a.S : most) * a.tiles_r + static_cast<int64_t>((a.T + kRows - 1) / kRows) * a.tiles_s;
  const int64_t grid = (tiles + kGemmXcds - 1) / kGemmXcds * kGemmXcds;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  switch (group) {
    case 32: int4_tile_kernel<MODE, 32><<<static_cast<unsigned>(grid), 256, 0, st>>>(a); break;
    case 64: int4_tile_kernel<MODE, 64><<<static_cast<unsigned>(grid), 256, 0, st>>>(a); break;
    default: int4_tile_kernel<MODE, 128><<<static_cast<unsigned>(grid), 256, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_int4(const Int4Args& a, int group, hipStream_t st) {
  switch (int4_kernel(MODE == kInt4GateUp, group, a.S, a.E)) {
    case Int4Kernel::kTiles: return launch_tiles4<MODE>(a, group, st);
    case Int4Kernel::kRows32: return launch_rows<MODE, 2>(a, group, st);
    default: return launch_rows<MODE, 1>(a, group, st);
  }
}

int grid_for(int64_t items) {
  const int64_t want = (items + 255) / 256;
  return static_cast<int>(want < 65536 ? want : 65536);
}

}  // namespace

hipError_t launch_quantize_int4(const bf16_t* src, uint8_t* dst, bf16_t* scales, int64_t count, int rows, int cols,
                                int group, hipStream_t st) {
  const int64_t nrows = count * rows;
  const int grid = grid_for(nrows * (cols / 8));
  switch (group) {
    case 32: quantize_int4_kernel<32><<<grid, 256, 0, st>>>(src, dst, scales, nrows, rows, cols); break;
    case 64: quantize_int4_kernel<64><<<grid, 256, 0, st>>>(src, dst, scales, nrows, rows, cols); break;
    default: quantize_int4_kernel<128><<<grid, 256, 0, st>>>(src, dst, scales, nrows, rows, cols); break;
  }
  return hipGetLastError();
}

hipError_t launch_pack_int4(const uint8_t* codes, uint8_t* dst, int64_t count, int rows, int cols, hipStream_t st) {
  pack_int4_kernel<<<grid_for(count * static_cast<int64_t>(rows) * cols / 8), 256, 0, st>>>(
      reinterpret_cast<const uint32_t*>(codes), dst, count, rows, cols);
  return hipGetLastError();
}

hipError_t launch_gate_up_int4(const moe_shape& s, int group, const bf16_t* x_perm, const int32_t* sorted_token,
                               const bf16_t* x, const int32_t* offsets, const uint8_t* wgu, const bf16_t* sgu,
                               const uint8_t* wsgu, const bf16_t* ssgu, bf16_t* h, hipStream_t st) {
  Int4Args a{};
  a.a_routed = x_perm ? x_perm : x;
  a.gather = x_perm ? nullptr : sorted_token;
  a.a_shared = x;
  a.w_routed = wgu;
  a.w_shared = wsgu;
  a.s_routed = sgu;
  a.s_shared = ssgu;
  a.out_routed = h;
  a.out_shared = h + static_cast<size_t>(s.T) * s.k * s.F;
  a.offsets = offsets;
  a.T = s.T;
  a.E = s.E;
  a.S = s.T * s.k;
  a.K = a.Ks = s.D;
  a.N = s.F;
  a.Ns = s.Fs;
  return launch_int4<kInt4GateUp>(a, group, st);
}

hipError_t launch_down_int4(const moe_shape& s, int group, const bf16_t* h, const int32_t* offsets,
                            const uint8_t* wd, const bf16_t* sd, const uint8_t* wsd, const bf16_t* ssd,
                            bf16_t* y_perm, bf16_t* y_shared, hipStream_t st) {
  Int4Args a{};
  a.a_routed = h;
  a.a_shared = h + static_cast<size_t>(s.T) * s.k * s.F;
  a.w_routed = wd;
  a.w_shared = wsd;
  a.s_routed = sd;
  a.s_shared = ssd;
  a.out_routed = y_perm;
  a.out_shared = y_shared;
  a.offsets = offsets;
  a.T = s.T;
  a.E = s.E;
  a.S = s.T * s.k;
  a.K = s.F;
  a.Ks = s.Fs;
  a.N = s.D;
  a.Ns = s.Fs > 0 ? s.D : 0;
  return launch_int4<kInt4Down>(a, group, st);
}

}  // namespace moe
