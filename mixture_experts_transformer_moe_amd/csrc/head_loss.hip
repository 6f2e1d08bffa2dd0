// Softmax cross entropy of the output head over a large vocabulary, without its
// logits, and the gradients of the hidden states and of the head's weights
// ("Laguna-M.1-base", Shape: vocabulary of 100352; the training step whose other
// end is the update).
//
//   z[t, v] = x_t w_v;  lse_t = log sum_v exp z[t, v];  loss_t = lse_t - z[t, y_t]
//   P[t, v] = (exp(z[t, v] - lse_t) - [v = y_t]) g_t;  dx = P W;  dW = P^T x
// A row whose target is outside the vocabulary takes no part.
//
// Forward: a tile of z stays in the accumulators; each row's maximum and sum over
// the tile's columns go out (8 bytes for 256 columns) and a second kernel joins
// them in a fixed order.  Backward: the vocabulary goes by in pieces; per piece z
// is computed again, P leaves the accumulators once as bf16, and two products follow,
// each with one operand read across its rows (gemm_nt.h): P W, and P^T with x
// transposed once (rows without part as zeros).  dx is summed over pieces in fp32.
// P in bf16 is the one rounding inside: 1.7e-3 of an entry, independent from entry to
// entry and common to the entry's whole row of W or x.  Held in more it would be a second
// product.  The target's entry, p - 1 from fp32, is most of a row's norm where the row
// knows its target: what its rounding lost is kept in fp32 and added to both products
// (333 x 1000 over 33001, rows that point at their target: 2.4e-3 of the gradients' norm
// without it, up to 3.4e-3 for single rows, 1.66e-3 with it, the outputs' own rounding;
// 3% of the time at 8192 x 4096 over 100352, 9% at 256 rows).  What other entries lose
// stays: where a row points at a rival of its target as well, the gradients are 2.1e-3
// off, single rows of dx up to 3.2e-3 and of dW up to 4.2e-3, and dW's rows of entries
// that are no row's target 2.3e-3 with either.
#include "head_loss.h"

#include "gemm_nt.h"
#include "head_plan.h"

namespace moe {
namespace {

typedef __attribute__((address_space(1))) unsigned char gbyte;
typedef __attribute__((address_space(1))) u32x4 gu32x4;

static_assert(kHeadStage == kNtBK, "the plan counts this product's stages");

using Rows32 = NtShape<1, 4, 1, 2>;
using Rows64 = NtShape<1, 4, 2, 2>;
using Mid = NtShape<2, 2, 2, 2>;
using Wide = NtShape<2, 2, 4, 4>;

template <class F>
void with_tile(Tile t, F&& f) {
  switch (t) {
    case kRows32: f(Rows32{}); break;
    case kRows64: f(Rows64{}); break;
    case kMid: f(Mid{}); break;
    default: f(Wide{}); break;
  }
}

// The bf16 tile of a wave (32 MB rows, 32 NB columns; value(m, n, r) gives register
// r of block (m, n), rounded) through its LDS, stored as whole row segments: rows
// below `rows`, columns below `cols` (whole pieces of 8).
template <class S, class F>
__device__ __forceinline__ void store_rows(bf16_t* out, size_t ld, int rows, int cols, unsigned char* stg, F&& value) {
  const int lane = threadIdx.x & 63;
  constexpr int kPieces = 4 * S::NB;                       // 16-byte pieces of a row
  constexpr int kRowB = 16 * kPieces;
  auto swz = [](int r) { return S::NB == 4 ? r & 15 : (r >> 1) & 7; };
#pragma unroll
  for (int m = 0; m < S::MB; ++m) {
#pragma unroll
    for (int n = 0; n < S::NB; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = lane & 31, c = 4 * n + q;
        uint2 v;
        v.x = pack_bf16x2(value(m, n, 4 * q), value(m, n, 4 * q + 1));
        v.y = pack_bf16x2(value(m, n, 4 * q + 2), value(m, n, 4 * q + 3));
        *reinterpret_cast<uint2*>(stg + r * kRowB + ((c ^ swz(r)) << 4) + 8 * (lane >> 5)) = v;
      }
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < kPieces / 2; ++i) {                // 64 pieces a store
      const int at = 64 * i + lane, r = at / kPieces, c = at % kPieces;
      const u32x4 v = *reinterpret_cast<const u32x4*>(stg + r * kRowB + ((c ^ swz(r)) << 4));
      if (32 * m + r < rows && 8 * c < cols)
        *(gu32x4*)((gbyte*)(out + static_cast<size_t>(32 * m + r) * ld + 8 * c)) = v;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
}

struct LogitArgs {
  const bf16_t* x;          // [T, D]
  const bf16_t* w;          // [V, D]
  const int32_t* target;    // [T]
  int T, D, V;
  int v0, v1;               // the columns of this launch
  int tiles_m, tiles_n;
  // forward
  float2* part;             // [T, parts]: maximum and sum of each column tile
  int parts;
  float* zt;                // [T]: the target's logit
  // backward
  const float* lse;
  const float* dloss;
  bf16_t* p;                // [T, ldp]
  float* rest;              // [T]: what the target's entry of P lost to bf16
  int ldp;
};

template <class S>
__device__ __forceinline__ void logits_tile(const LogitArgs& g, unsigned char* smem, int& t0, int& v0, f32x16 (&acc)[S::MB][S::NB]) {
  int tm, tn, z;
  nt_tile(blockIdx.x, g.tiles_m, g.tiles_n, 1, tm, tn, z);
  t0 = tm * S::BM;
  v0 = g.v0 + tn * S::BN;
  const NtOperand a{g.x + static_cast<size_t>(t0) * g.D, g.D, g.T - t0};
  const NtOperand b{g.w + static_cast<size_t>(v0) * g.D, g.D, g.V - v0};
  gemm_nt<S>(a, b, g.D, smem, acc, [] {});
}

template <class S>
__global__ __launch_bounds__(kNtThreads, S::kLds > 80 * 1024 ? 1 : 2) void head_stats_kernel(LogitArgs g) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[S::kLds];
  f32x16 acc[S::MB][S::NB];
  int t0, v0;
  logits_tile<S>(g, smem, t0, v0, acc);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave / S::WC, wc = wave % S::WC;
  float2* red = reinterpret_cast<float2*>(smem);           // [WC][BM]
  const int vw = v0 + 32 * S::NB * wc + 4 * (lane >> 5);   // the lane's first column
  const bool edge = v0 + S::BN > g.V;
#pragma unroll
  for (int m = 0; m < S::MB; ++m) {
    const int row = 32 * (S::MB * wr + m) + (lane & 31), t = t0 + row;
    const int y = g.target[min(t, g.T - 1)];
    const bool here = t < g.T && y >= v0 && y < v0 + S::BN && y < g.V;
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < S::NB; ++n) {
      asm volatile("" : "+a"(acc[m][n]));                  // one block's accumulators at a time
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int v = vw + 32 * n + 8 * (r >> 2) + (r & 3);
        if (edge && v >= g.V) acc[m][n][r] = -INFINITY;
        top = fmaxf(top, acc[m][n][r]);
      }
      if (here) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (vw + 32 * n + 8 * (r >> 2) + (r & 3) == y) g.zt[t] = acc[m][n][r];
      }
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    const float from = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < S::NB; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) sum += __expf(acc[m][n][r] - from);
    sum += __shfl_xor(sum, 32);
    if (lane < 32) red[wc * S::BM + row] = make_float2(top, sum);
  }
  __syncthreads();
  for (int row = tid; row < S::BM; row += kNtThreads) {
    if (t0 + row >= g.T) break;
    float2 all = red[row];
#pragma unroll
    for (int c = 1; c < S::WC; ++c) {
      const float2 o = red[c * S::BM + row];
      const float top = fmaxf(all.x, o.x), from = top == -INFINITY ? 0.0f : top;
      all = make_float2(top, all.y * __expf(all.x - from) + o.y * __expf(o.x - from));
    }
    g.part[static_cast<size_t>(t0 + row) * g.parts + (v0 - g.v0) / S::BN] = all;
  }
}

// One wave a row joins the tiles' maxima and sums.
__global__ __launch_bounds__(256) void head_join_kernel(const float2* part, int parts, const float* zt,
                                                        const int32_t* target, int T, int V, float* loss, float* lse) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int y = target[t];
  if (y < 0 || y >= V) {
    if (lane == 0) loss[t] = lse[t] = 0.0f;
    return;
  }
  const float2* p = part + static_cast<size_t>(t) * parts;
  float top = -INFINITY;
  for (int i = lane; i < parts; i += 64) top = fmaxf(top, p[i].x);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float from = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  for (int i = lane; i < parts; i += 64) sum += p[i].y * __expf(p[i].x - from);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) {
    const float l = logf(sum);
    lse[t] = from + l;
    loss[t] = (from - zt[t]) + l;                          // exact where the target is the largest
  }
}

template <class S>
__global__ __launch_bounds__(kNtThreads, S::kLds > 80 * 1024 ? 1 : 2) void head_probs_kernel(LogitArgs g) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[S::kLds];
  f32x16 acc[S::MB][S::NB];
  int t0, v0;
  logits_tile<S>(g, smem, t0, v0, acc);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / S::WC, wc = wave % S::WC;
  const int tw = t0 + 32 * S::MB * wr, vw = v0 + 32 * S::NB * wc;   // the wave's first row and column
  // P over z, in the accumulators
#pragma unroll
  for (int m = 0; m < S::MB; ++m) {
    const int t = tw + 32 * m + (lane & 31), tc = min(t, g.T - 1);
    const int y = g.target[tc];
    const bool takes = t < g.T && y >= 0 && y < g.V;
    const float lse = g.lse[tc], w = g.dloss[tc];
    float mine = 0.0f;                                     // the target's entry, where this lane holds it
#pragma unroll
    for (int n = 0; n < S::NB; ++n) {
      asm volatile("" : "+a"(acc[m][n]));
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int v = vw + 32 * n + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        float p = __expf(acc[m][n][r] - lse);
        if (v == y) p -= 1.0f;
        p = takes && v < g.V ? p * w : 0.0f;
        mine = v == y ? p : mine;
        acc[m][n][r] = p;
      }
      asm volatile("" : "+a"(acc[m][n]));
    }
    const int at = y - vw;
    if (takes && at >= 0 && at < 32 * S::NB && (at >> 2 & 1) == lane >> 5)
      g.rest[t] = mine - bf16_to_f32(f32_to_bf16(mine));
  }
  store_rows<S>(g.p + static_cast<size_t>(tw) * g.ldp + (vw - g.v0), g.ldp, g.T - tw, g.ldp - (vw - g.v0),
                smem + wave * 2048 * S::NB, [&](int m, int n, int r) { return acc[m][n][r]; });
}

// dx: A = P [M, lda], B = W [depth, N]; dW (DW): A = P [depth, lda], B = x transposed
// [N, ldb].  What is not transposed holds zeros past the reduction's end.
struct ProductArgs {
  const bf16_t* a;
  const bf16_t* b;
  int M, N, K, lda, ldb;    // K a multiple of 64
  int depth;
  int tiles_m, tiles_n, parts;
  bf16_t* out;              // [M, N] bf16
  float* sums;              // where the reduction comes in parts or pieces: fp32, as the
                            // accumulators lie (whole kilobytes a wave and load)
  int add, last;            // added to what sums holds; the last piece, straight to out
  // the target's entries of P, whose rounding is made good
  const int32_t* target;    // [T]
  const float* rest;        // [T]
  int T, v0, v1;            // the piece's columns of P
  const bf16_t* x;          // DW: [T, N], and its rows in order of their targets (order_rows)
  const int32_t* order;
  const int32_t* order_at;
  int order_groups;
};

// where the sums of a wave's tile start, in float4
template <class S>
__device__ __forceinline__ size_t sums_at(int tile, int wave) {
  return (static_cast<size_t>(tile) * 4 + wave) * (S::MB * S::NB * 256);
}

// dW: the entries from .. to - 1 of a tile's list, 64 at a time as a stage of the
// reduction.  Their rows of x go to LDS by direct loads, two stages deep, laid out as
// gemm_nt.h has an operand that is read across its rows; the other operand holds an
// entry's value where its column is the lane's.  Frequent targets and small
// vocabularies make such lists: 16384 x 2048 over 500 lists of 4096, whose gradients
// take 357 us (1179 with 16 entries at a time by ordinary loads), 8192 x 4096 over 8192
// of 256, 1371 us (1572).
template <class S>
__device__ __forceinline__ void add_listed(const ProductArgs& g, int from, int to, int n0, unsigned char* smem,
                                           f32x16 (&acc)[S::MB][S::NB]) {
  constexpr int kList = 64, kBuf = kList * S::BN * 2, kLoads = S::BN / 32, kUnits = S::BN / 8;
  static_assert(2 * kBuf + 4 * kList * 4 <= S::kLds, "two stages and each wave's entries");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / S::WC, wc = wave % S::WC;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  uint32_t* own = reinterpret_cast<uint32_t*>(smem + 2 * kBuf) + kList * wave;
  // lane l's entry of the stage at e (past the list's end: its last, with nothing to add)
  auto entry_at = [&](int e) { return g.order[min(e + lane, to - 1)]; };
  auto rest_at = [&](int entry, int e) { return e + lane < to ? g.rest[entry >> 8] : 0.0f; };
  auto issue = [&](int entry, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int r = 64 / kUnits * (kLoads * wave + q) + lane / kUnits;
      const int t = __shfl(entry, r) >> 8;
      const int col = min(8 * ((lane % kUnits) ^ (4 * (r & 3))), g.N - n0 - 8);
      dma16(g.x + static_cast<size_t>(t) * g.N + n0 + col,
            __builtin_amdgcn_readfirstlane(lds0 + buf * kBuf + (kLoads * wave + q) * 1024));
    }
  };
  int entry = entry_at(from), next = entry_at(from + kList), buf = 0;
  issue(entry, 0);
  float rest = rest_at(entry, from);
  for (int e = from; e < to; e += kList, buf ^= 1) {
    own[lane] = static_cast<uint32_t>(entry & (S::BM - 1)) << 16 | f32_to_bf16(rest);
    // the stage has landed, and every wave has read the one before
    __builtin_amdgcn_s_waitcnt(nt_lgkm_only(0));
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (e + kList < to) {
      entry = next;
      issue(entry, buf ^ 1);
      rest = rest_at(entry, e + kList);
      next = entry_at(e + 2 * kList);
    }
#pragma unroll
    for (int s = 0; s < kList / 16; ++s) {
      u32x4 x[S::NB];
#pragma unroll
      for (int n = 0; n < S::NB; ++n)
        x[n] = nt_read_step(lds0 + buf * kBuf + nt_tr_at(lane, S::NB * wc + n, kUnits), S::BN * 2, s);
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = own[16 * s + 8 * (lane >> 5) + j];
#pragma unroll
      for (int m = 0; m < S::MB; ++m) {
        const uint32_t col = 32 * (S::MB * wr + m) + (lane & 31);
        u32x4 r;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[j] = (w[2 * j] >> 16 == col ? w[2 * j] & 0xffffu : 0u) | (w[2 * j + 1] >> 16 == col ? w[2 * j + 1] << 16 : 0u);
#pragma unroll
        for (int n = 0; n < S::NB; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x[n]), __builtin_bit_cast(bf16x8, r),
                                                              acc[m][n], 0, 0, 0);
      }
    }
  }
  __syncthreads();                                            // (the waves' stores go through the buffers)
}

template <class S, bool DW, bool SUMS>
__global__ __launch_bounds__(kNtThreads, S::kLds > 80 * 1024 ? 1 : 2) void head_product_kernel(ProductArgs g) {
  __shared__ __attribute__((aligned(1024))) unsigned char smem[S::kLds];
  int tm, tn, z;
  nt_tile(blockIdx.x, g.tiles_m, g.tiles_n, g.parts, tm, tn, z);
  const int nk = g.K / kNtBK;
  const int k0 = static_cast<int>(static_cast<int64_t>(nk) * z / g.parts), k1 = static_cast<int>(static_cast<int64_t>(nk) * (z + 1) / g.parts);
  const int m0 = tm * S::BM, n0 = tn * S::BN;
  f32x16 acc[S::MB][S::NB];
  const size_t kat = static_cast<size_t>(k0) * kNtBK;
  const int depth = g.depth - k0 * kNtBK;
  const NtOperand a{DW ? g.a + kat * g.lda + m0 : g.a + static_cast<size_t>(m0) * g.lda + kat, g.lda,
                    (DW ? g.lda : g.M) - m0, depth};
  const NtOperand b{DW ? g.b + static_cast<size_t>(n0) * g.ldb + kat : g.b + kat * g.ldb + n0, g.ldb, g.N - n0, depth};
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / S::WC, wc = wave % S::WC;
  const int mw = m0 + 32 * S::MB * wr, nw = n0 + 32 * S::NB * wc;

  // What the targets' entries of P lost, read ahead of the reduction.  DW: the first 16
  // of the tile's list of rows with a target among its columns, as 16 more values of
  // the reduction, in bf16 (a target's entry then has 16 bits).
  struct Lost {
    int row[8];             // the column of P in the tile, -1: none
    float rest[8];
    bf16x8 x[S::NB];
  } lost;
  int list_at = 0, list_end = 0;
  // (scalar loads: a vector load's wait would count the stages under way)
  typedef const __attribute__((address_space(4))) int32_t* Scalars;
  auto load_lost = [&]() __attribute__((always_inline)) {
    int entries[16];                                       // (past the list's end: still in the workspace)
#pragma unroll
    for (int i = 0; i < 16; ++i) entries[i] = ((Scalars)(g.order))[list_at + i];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = list_at + 8 * (lane >> 5) + j;
      const int entry = i < list_end ? (lane < 32 ? entries[j] : entries[8 + j]) : -1;
      const int t = entry < 0 ? 0 : entry >> 8;
      lost.row[j] = entry < 0 ? -1 : entry & (S::BM - 1);
      lost.rest[j] = entry < 0 ? 0.0f : g.rest[t];
#pragma unroll
      for (int n = 0; n < S::NB; ++n) {
        const int col = nw + 32 * n + (lane & 31);
        const bool in = entry >= 0 && col < g.N;
        lost.x[n][j] = __builtin_bit_cast(__bf16, in ? g.x[static_cast<size_t>(t) * g.N + col] : bf16_t{0});
      }
    }
  };
  // (dx: each row's target and what its entry lost, where this piece holds it)
  int to[S::MB];
  float rest[S::MB];
  gemm_nt<S, DW, !DW>(a, b, (k1 - k0) * kNtBK, smem, acc, [&]() __attribute__((always_inline)) {
    if constexpr (DW) {
      const int first = (g.v0 + m0) / kOrderCols;
      list_at = ((Scalars)(g.order_at))[first];
      list_end = ((Scalars)(g.order_at))[min(first + S::BM / kOrderCols, g.order_groups)];
      if (list_at < list_end) load_lost();
    } else {
#pragma unroll
      for (int m = 0; m < S::MB; ++m) {
        const int t = mw + 32 * m + (lane & 31);
        const int v = z == 0 && t < g.T ? g.target[t] : -1;
        to[m] = v >= g.v0 && v < g.v1 ? v - g.v0 : -1;
        rest[m] = to[m] >= 0 ? g.rest[t] : 0.0f;
      }
    }
  });
  if constexpr (DW) {
    if (list_at < list_end) {
      bf16x8 r[S::MB];
#pragma unroll
      for (int m = 0; m < S::MB; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          r[m][j] = __builtin_bit_cast(
              __bf16, lost.row[j] == 32 * (S::MB * wr + m) + (lane & 31) ? f32_to_bf16(lost.rest[j]) : bf16_t{0});
#pragma unroll
      for (int m = 0; m < S::MB; ++m)
#pragma unroll
        for (int n = 0; n < S::NB; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lost.x[n], r[m], acc[m][n], 0, 0, 0);
      if (list_at + 16 < list_end) add_listed<S>(g, list_at + 16, list_end, n0, smem, acc);
    }
  } else if (z == 0) {
    // row t takes rest[t] times its target's row of W
#pragma unroll
    for (int m = 0; m < S::MB; ++m) {
      const bf16_t* row = g.b + static_cast<size_t>(max(to[m], 0)) * g.ldb;
#pragma unroll
      for (int n0 = 0; n0 < S::NB; n0 += 2) {
        uint2 w[2][4];                                     // (two blocks' loads at a time)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = nw + 32 * (n0 + i) + 8 * q + 4 * (lane >> 5);
            w[i][q] = to[m] >= 0 && col < g.N ? *reinterpret_cast<const uint2*>(row + col) : make_uint2(0u, 0u);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f32x16& c = acc[m][n0 + i];
          if constexpr (S::MB * S::NB > 8) asm volatile("" : "+a"(c));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            c[4 * q] = fmaf(rest[m], __uint_as_float(w[i][q].x << 16), c[4 * q]);
            c[4 * q + 1] = fmaf(rest[m], __uint_as_float(w[i][q].x & 0xffff0000u), c[4 * q + 1]);
            c[4 * q + 2] = fmaf(rest[m], __uint_as_float(w[i][q].y << 16), c[4 * q + 2]);
            c[4 * q + 3] = fmaf(rest[m], __uint_as_float(w[i][q].y & 0xffff0000u), c[4 * q + 3]);
          }
          if constexpr (S::MB * S::NB > 8) asm volatile("" : "+a"(c));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  bf16_t* out = g.out + static_cast<size_t>(mw) * g.N + nw;
  auto rounded = [&]() __attribute__((always_inline)) {
    store_rows<S>(out, g.N, g.M - mw, g.N - nw, smem + wave * 2048 * S::NB, [&](int m, int n, int r) { return acc[m][n][r]; });
  };
  if constexpr (!SUMS) {
    rounded();
  } else {
    float4* sums = reinterpret_cast<float4*>(g.sums) + sums_at<S>((z * g.tiles_m + tm) * g.tiles_n + tn, wave) + lane;
#pragma unroll
    for (int m = 0; m < S::MB; ++m)
#pragma unroll
      for (int n = 0; n < S::NB; ++n) {
        if constexpr (S::MB * S::NB > 8) asm volatile("" : "+a"(acc[m][n]));   // one block at a time
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float4* at = sums + ((m * S::NB + n) * 4 + q) * 64;
          float4 v = make_float4(acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]);
          if (g.add) {
            const float4 o = *at;
            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
          }
          if (g.last) {
            acc[m][n][4 * q] = v.x;
            acc[m][n][4 * q + 1] = v.y;
            acc[m][n][4 * q + 2] = v.z;
            acc[m][n][4 * q + 3] = v.w;
          } else {
            *at = v;
          }
        }
      }
    if (g.last) rounded();
  }
}

// dx from the parts of its sum, in their order: four values a thread
template <class S>
__global__ __launch_bounds__(256) void head_round_kernel(ProductArgs g) {
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;   // (a workgroup: one accumulator block)
  const int block = blockIdx.x % (S::MB * S::NB), wave = blockIdx.x / (S::MB * S::NB) % 4;
  const int tile = blockIdx.x / (4 * S::MB * S::NB);
  const int m = block / S::NB, n = block % S::NB;
  const int row = tile / g.tiles_n * S::BM + 32 * (S::MB * (wave / S::WC) + m) + (lane & 31);
  const int col = tile % g.tiles_n * S::BN + 32 * (S::NB * (wave % S::WC) + n) + 8 * q + 4 * (lane >> 5);
  if (row >= g.M || col >= g.N) return;
  const float4* sums = reinterpret_cast<const float4*>(g.sums);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8                                            // (few waves: loads ahead of their additions, 7.0 us for 9.1)
  for (int z = 0; z < g.parts; ++z) {
    const float4 o = sums[sums_at<S>(z * g.tiles_m * g.tiles_n + tile, wave) + (block * 4 + q) * 64 + lane];
    v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
  }
  *reinterpret_cast<uint2*>(g.out + static_cast<size_t>(row) * g.N + col) =
      make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// The rows of a batch by the 128-column group of their target, in order within it:
// order[i] = row << 8 | target mod 256, order_at[g] the first of group g.  A workgroup
// a group: the targets of lower groups give its place, then each wave writes the
// matches of its quarter of the batch.
__device__ __forceinline__ void order_rows(int group, const int32_t* target, int T, int V, int32_t* order,
                                           int32_t* order_at) {
  __shared__ int less_of[4], own_of[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int v0 = group * kOrderCols, v1 = min(v0 + kOrderCols, V);
  const int quarter = (T + 255) / 256 * 64;
  const int from = wave * quarter, to = min(from + quarter, T);
  int less = 0, own = 0;
#pragma unroll 8
  for (int t = from + lane; t < to; t += 64) {
    const int y = target[t];
    less += y >= 0 && y < v0;
    own += y >= v0 && y < v1;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    less += __shfl_xor(less, o);
    own += __shfl_xor(own, o);
  }
  if (lane == 0) {
    less_of[wave] = less;
    own_of[wave] = own;
  }
  __syncthreads();
  const int start = less_of[0] + less_of[1] + less_of[2] + less_of[3];
  int at = start, all = start;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) at += own_of[w];
    all += own_of[w];
  }
  if (threadIdx.x == 0) {
    order_at[group] = start;
    if (v1 == V) order_at[group + 1] = all;
  }
  if (own_of[wave] == 0) return;
  for (int i = from; i < to; i += 64) {
    const int t = i + lane;
    const int y = t < to ? target[t] : -1;
    const bool here = y >= v0 && y < v1;
    const uint64_t mask = __ballot(here);
    if (here) order[at + __popcll(mask & ((uint64_t{1} << lane) - 1))] = t << 8 | (y & 255);
    at += __popcll(mask);
  }
}

// dst [cols, ldd] = src [rows, cols]^T in 64 x 64 tiles; columns of dst from rows to
// ldd (a multiple of 64) are zero, and so are those of rows whose target is outside
// the vocabulary (what stands in them may be no number)
__device__ __forceinline__ void transpose_rows(int block, const bf16_t* src, int rows, int cols, bf16_t* dst, int ldd,
                                               const int32_t* target, int V) {
  __shared__ __attribute__((aligned(16))) bf16_t tile[64][72];
  const int tid = threadIdx.x;
  const int tr = ldd / 64;
  const int r0 = block % tr * 64, c0 = block / tr * 64;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 32 * i + tid / 8, c = tid % 8 * 8;
    u32x4 v = {0u, 0u, 0u, 0u};
    bool takes = r0 + r < rows && c0 + c < cols;
    if (takes) {
      const int y = target[r0 + r];
      takes = y >= 0 && y < V;
    }
    if (takes) v = *reinterpret_cast<const u32x4*>(src + static_cast<size_t>(r0 + r) * cols + c0 + c);
    *reinterpret_cast<u32x4*>(&tile[r][c]) = v;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = 32 * i + tid / 8, r = tid % 8 * 8;
    if (c0 + c >= cols) continue;
    union {
      u32x4 v;
      bf16_t e[8];
    } o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o.e[j] = tile[r + j][c];
    *reinterpret_cast<u32x4*>(dst + static_cast<size_t>(c0 + c) * ldd + r0 + r) = o.v;
  }
}

// what dW's products need of the batch, in one launch
__global__ __launch_bounds__(256) void head_prepare_kernel(const bf16_t* x, const int32_t* target, int T, int D, int V,
                                                           int order_groups, int32_t* order, int32_t* order_at,
                                                           bf16_t* xt, int ldt) {
  const int b = blockIdx.x;
  if (b < order_groups) order_rows(b, target, T, V, order, order_at);
  else transpose_rows(b - order_groups, x, T, D, xt, ldt, target, V);
}

__global__ __launch_bounds__(256) void head_zero_kernel(u32x4* out, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256)
    out[i] = u32x4{0u, 0u, 0u, 0u};
}

unsigned blocks_for(int64_t items) {
  const int64_t want = (items + 255) / 256;
  return static_cast<unsigned>(want < 4096 ? want : 4096);
}

template <class S>
void launch_stats(LogitArgs g, hipStream_t st) {
  g.parts = (g.V + S::BN - 1) / S::BN;
  g.tiles_m = (g.T + S::BM - 1) / S::BM;
  g.tiles_n = (g.v1 - g.v0 + S::BN - 1) / S::BN;
  head_stats_kernel<S><<<g.tiles_m * g.tiles_n, kNtThreads, 0, st>>>(g);
}

template <class S>
void launch_probs(LogitArgs g, hipStream_t st) {
  g.tiles_m = (g.T + S::BM - 1) / S::BM;
  g.tiles_n = (g.v1 - g.v0 + S::BN - 1) / S::BN;
  head_probs_kernel<S><<<g.tiles_m * g.tiles_n, kNtThreads, 0, st>>>(g);
}

template <class S, bool DW>
void launch_product(ProductArgs g, hipStream_t st) {
  g.tiles_m = (g.M + S::BM - 1) / S::BM;
  g.tiles_n = (g.N + S::BN - 1) / S::BN;
  const unsigned grid = g.tiles_m * g.tiles_n * g.parts;
  if (!DW && g.sums) head_product_kernel<S, DW, !DW><<<grid, kNtThreads, 0, st>>>(g);
  else head_product_kernel<S, DW, false><<<grid, kNtThreads, 0, st>>>(g);
}

template <class S>
void launch_round(ProductArgs g, hipStream_t st) {
  g.tiles_m = (g.M + S::BM - 1) / S::BM;
  g.tiles_n = (g.N + S::BN - 1) / S::BN;
  head_round_kernel<S><<<g.tiles_m * g.tiles_n * 4 * S::MB * S::NB, 256, 0, st>>>(g);
}

}  // namespace

size_t head_loss_workspace_bytes(int64_t rows, int cols, int vocab) { return workspace_bound(rows, cols, vocab); }

hipError_t launch_head_loss_forward(int rows, int cols, int vocab, const bf16_t* x, const bf16_t* w,
                                    const int32_t* target, float* loss, float* lse, void* workspace, hipStream_t st) {
  LogitArgs g{};
  g.x = x;
  g.w = w;
  g.target = target;
  g.T = rows;
  g.D = cols;
  g.V = vocab;
  g.v1 = vocab;
  const Tile t = tile_of_logits(rows, vocab, cols);
  g.parts = (vocab + cols_of(t) - 1) / cols_of(t);
  g.part = static_cast<float2*>(workspace);
  g.zt = reinterpret_cast<float*>(g.part + static_cast<size_t>(rows) * g.parts);
  with_tile(t, [&](auto s) { launch_stats<decltype(s)>(g, st); });
  if (hipError_t e = hipGetLastError()) return e;
  head_join_kernel<<<(rows + 3) / 4, 256, 0, st>>>(g.part, g.parts, g.zt, target, rows, vocab, loss, lse);
  return hipGetLastError();
}

hipError_t launch_head_loss_backward(int rows, int cols, int vocab, const bf16_t* x, const bf16_t* w,
                                     const int32_t* target, const float* lse, const float* dloss, bf16_t* dx,
                                     bf16_t* dw, void* workspace, hipStream_t st) {
  if (rows == 0) {
    const int64_t n = static_cast<int64_t>(vocab) * cols / 8;
    if (dw) head_zero_kernel<<<blocks_for(n), 256, 0, st>>>(reinterpret_cast<u32x4*>(dw), n);
    return hipGetLastError();
  }
  const Plan q = plan(rows, cols, vocab);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  bf16_t* p = reinterpret_cast<bf16_t*>(ws + q.p);
  bf16_t* xt = reinterpret_cast<bf16_t*>(ws + q.xt);
  float* sums = reinterpret_cast<float*>(ws + q.dx);
  float* rest = reinterpret_cast<float*>(ws + q.rest);
  int32_t* order = reinterpret_cast<int32_t*>(ws + q.order);
  int32_t* order_at = reinterpret_cast<int32_t*>(ws + q.order_at);
  const int order_groups = (vocab + kOrderCols - 1) / kOrderCols;
  const int col_tiles = (cols + 63) / 64;
  if (dw)
    head_prepare_kernel<<<order_groups + col_tiles * (q.ldt / 64), 256, 0, st>>>(x, target, rows, cols, vocab, order_groups,
                                                                                order, order_at, xt, q.ldt);
  for (int v0 = 0; v0 < vocab; v0 += q.piece) {
    const int width = piece_width(q, v0, vocab), v1 = v0 + width;
    const int ldp = up(width, kHeadStage);
    LogitArgs g{};
    g.x = x;
    g.w = w;
    g.target = target;
    g.T = rows;
    g.D = cols;
    g.V = vocab;
    g.v0 = v0;
    g.v1 = v1;
    g.lse = lse;
    g.dloss = dloss;
    g.p = p;
    g.rest = rest;
    g.ldp = ldp;
    ProductArgs base{};
    base.target = target;
    base.rest = rest;
    base.x = x;
    base.T = rows;
    base.order = order;
    base.order_at = order_at;
    base.order_groups = order_groups;
    base.v0 = v0;
    base.v1 = v1;
    with_tile(tile_of_logits(rows, width, cols), [&](auto s) { launch_probs<decltype(s)>(g, st); });
    if (dw) {
      ProductArgs d = base;
      d.a = p;
      d.b = xt;
      d.M = width;
      d.N = cols;
      d.K = d.ldb = q.ldt;
      d.lda = ldp;
      d.depth = rows;
      d.parts = 1;
      d.out = dw + static_cast<size_t>(v0) * cols;
      if (tile_of_dw(q, width, cols) == kMid) launch_product<Mid, true>(d, st);
      else launch_product<Wide, true>(d, st);
    }
    if (dx) {
      ProductArgs d = base;
      d.a = p;
      d.b = w + static_cast<size_t>(v0) * cols;
      d.M = rows;
      d.N = cols;
      d.K = ldp;
      d.lda = ldp;
      d.ldb = cols;
      d.depth = width;                                     // (P's columns past it are zeros)
      d.parts = parts_of_dx(q, width);
      d.out = dx;
      d.sums = q.sums ? sums : nullptr;
      d.add = v0 > 0;
      d.last = v1 == vocab && q.parts == 1;
      with_tile(q.tile, [&](auto s) { launch_product<decltype(s), false>(d, st); });
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (dx && q.parts > 1) {
    ProductArgs d{};
    d.M = rows;
    d.N = cols;
    d.parts = q.parts;
    d.out = dx;
    d.sums = sums;
    with_tile(q.tile, [&](auto s) { launch_round<decltype(s)>(d, st); });
  }
  return hipGetLastError();
}

}  // namespace moe
