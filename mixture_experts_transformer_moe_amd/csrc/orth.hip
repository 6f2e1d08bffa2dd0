// Orthogonalised update of weight matrices (the direction of the Muon
// optimiser): Newton-Schulz steps on the matrix cores, batched over experts.
//
// Per matrix u (the gradient, or gradient and momentum joined), taken with its
// short side first (m <= n; a tall matrix is read and written transposed):
//   x_0 = u / (|u|_F + eps),   x <- (a I + b R + c R^2) x,  R = x x^T,
// `steps` times, out = scale * x in bf16.
//
// Grouping.  The polynomial Q(R) of a step commutes with R, so the next step's
// Gram matrix is R' = Q R Q, and two steps apply as one product:
//   x <- Q2(R') Q1(R) x.
// With symmetric products computing one triangle, the pair costs
// 3 m^2 n + 5 m^3 flops against 6 m^2 n + 2 m^3 one by one, so the first two
// steps are taken together where the matrix is wide (n >= 1.5 m).  Later steps
// are not: R' holds R's small eigenvalues only to its rounding, which does not
// matter while Q(R) acts on them as a I, but does once the spectrum is flat.
// Nor are three, nor those of a small matrix (m < 256), whose roundings average
// over few terms.  Error against 64 bits, relative in norm, of rank-deficient
// gradients (the output's own rounding to bf16 is 1.7e-3 of each):
//                                         1+1+1+1+1  2+1+1+1  3+1+1   3+2
//   1024 x 2048, rank 128                 1.9e-3     1.9e-3   2.0e-3  2.3e-3
//   256 x 1024, rank 1 and noise of 1e-3  1.9e-3     2.0e-3   3.2e-3  3.1e-3
//   32 x 32, rank 16                      2.2e-3     2.4e-3   5.3e-3  5.6e-3
//
// Numbers.  Products run on fp16 operands with fp32 accumulation: singular
// directions far below the largest are amplified by a^5 = 485, and bf16's 8
// bits would add noise of 1% to 30% of the result.  Two parts are kept finer,
// at no product's cost:
//   * a symmetric matrix is stored as M + diag(d): d the diagonal rounded to
//     fp16, M the rest in fp16 (on the diagonal what d leaves).  (M + d)(N + e) =
//     M N + d_i N_ij + M_ij e_j + d_i e_i is joined in fp32 in the epilogue.
//     The polynomial of a nearly null direction is a I, whose rounding would
//     otherwise be the largest error;
//   * x is stored as fp16 hi + lo (22 bits).  M x and diag(d) x read hi (the
//     latter as MFMAs with a diagonal operand, in the stage that holds the
//     rows), the epilogue adds g_i lo_ij, g_i near a or d_i (LowGain below; with
//     d_i throughout 32 x 32 of rank 16 is 3.8e-3 off, after 8 steps 3e-2).  The x
//     before the last step has no low part: what its rounding adds is amplified
//     by a at most (second line of the table above 1.7e-3 -> 2.0e-3; without it
//     in the last two 2.9e-3).
// Powers of two keep fp16 away from its subnormals: x and R are stored times
// 2^12 (|x|, |R| < 2), Q and Q2 Q1 times 2^8 (|Q2 Q1| <= a^2 = 12).
//
// Layout.  Every matrix of the workspace is a grid of 32 x 16 blocks of 1 KB
// (row-block major), a block holding the 64 lanes' 16-byte runs of a
// v_mfma_f32_32x32x16_f16 operand: element (r, c) of a block sits in run
// (r ^ 4 h ^ 8 o) + 32 h, h = c / 8, o the parity of the block's column.
//   * a product's stage (32 values of K) is whole kilobytes, loaded straight
//     into LDS and read as operands at lane order, without a bank conflict;
//   * x is the transposed operand of the last product of a group (K = its
//     rows): the transposing LDS read takes it from the same blocks, and the
//     two XORs put its 8-byte pieces into distinct banks;
//   * an accumulator block leaves as two whole blocks after one lane-pair
//     swap; its mirror image (symmetric products) goes through 2 KB of LDS and
//     the same transposing read.
// Rows and columns are padded with zeros to multiples of 32 (at least 128):
// zero rows stay zero, and the padded diagonal of Q meets zero rows of x.
#include <type_traits>

#include "lds_dma.h"

namespace moe {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;   // the quintic's coefficients
constexpr float kSX = 4096.0f;        // stored scale of x and R
constexpr float kSQ = 256.0f;         // stored scale of Q and products of Qs
constexpr int kOThreads = 256;        // 4 waves, 2 x 2
constexpr int kOBK = 32;              // K per stage
constexpr int kStages = 4;            // stages of the ring
constexpr int kOXcds = 8;
constexpr int kMinPad = 128;          // smallest padded side: a tile has at least kStages stages

// kFinal: x <- P x into the caller's matrix, x without a low part (kFinalLo: with)
enum { kGram = 0, kPoly = 1, kMul = 2, kApply = 3, kFinal = 4, kFinalLo = 5 };

// What multiplies x's low part in x <- P x, P the polynomials of k steps.  The
// product itself reads x's high part, so with g_i for the low part x is off by
//   (P - a^k I) lo + (a^k - g_i) lo.
// The first lies in the columns' span of x, since P - a^k I = b R + ..., and stays
// as small as it is.  The second does not: each step to follow multiplies by a
// what lies outside the span.  So g_i = a^k while steps follow.  With two to
// follow the first part counts as well, most of all for a matrix near a diagonal
// one, which d_i would have exact.  By then P = a^k I - K, K near kappa times the
// projector on the span, so K_ii / kappa tells how much of row i's unit vector the
// span holds:
//   e_i = a^k - d_i = K_ii,  g_i = d_i + e_i (1 - e_i / kappa).
// In the last two products nothing is amplified any more, and g_i = d_i.  (Off by,
// with d_i throughout / a^k also with two to follow / as here: 32 x 32 of rank 16
// 3.8e-3 / 2.1e-3 / 2.2e-3, 333 x 1001 of rank 100 2.5e-3 / 2.0e-3 / 2.0e-3, the
// largest element's error of a diagonal matrix over three decades, in half steps of
// bf16, 1.56 / 1.91 / 1.56.)
struct LowGain {
  float a, w, k;            // a^k; 1, or 0 for g = d; 1 / kappa, or 0 for g = a^k
  __device__ __forceinline__ float operator()(float d) const {
    const float e = a - d;
    return fmaf(fmaxf(fmaf(-e, k, w), 0.0f), e, d);
  }
};

__host__ __device__ __forceinline__ LowGain low_gain(int taken, int after) {
  constexpr float kKappa = kB * kB / (4.0f * kC);   // a - min Q
  const float more = taken == 2 ? kA : 1.0f;
  return {kA * more, after < 2 ? 0.0f : 1.0f, after == 2 ? 1.0f / (kKappa * more) : 0.0f};
}

struct OrthJob {
  const _Float16* p;        // row operand, [rows / 32][K / 16] blocks
  const _Float16* q;        // column operand; kApply, kFinal, kFinalLo: x hi, [K / 32][n / 16] blocks
  const _Float16* lo;       // kApply / kFinalLo: x lo
  const float* dp;          // diagonals of p and q
  const float* dq;
  _Float16* out;            // kFinal: unused
  _Float16* out_lo;         // kApply: the low part, or null
  float* dout;
  float sp, sq, so;         // stored scales of p, q and out
  LowGain low;              // kApply: what x's low part is multiplied by
};

struct OrthArgs {
  OrthJob job;
  int count;                // matrices
  int mb, nb;               // row blocks (32) of the output, column blocks (32)
  int K;                    // reduction length
  int64_t p_stride, q_stride, out_stride;   // elements between matrices
  int d_stride;
  // kFinal: the caller's matrix
  bf16_t* user;
  int rows, cols, tall;     // tall: the caller's matrix is the transpose
  float scale;
};

// byte offset of the run of row r, half h (columns 8h..8h+7) in a block whose
// column block has parity o
__device__ __forceinline__ int run_off(int r, int h, int o) {
  return ((r ^ (h << 2) ^ (o << 3)) << 4) + (h << 9);
}

__device__ __forceinline__ void dma_run(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(voff), "s"(base), "s"(lds)
               : "memory", "m0");
}

template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v)));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32)));
  return reinterpret_cast<T*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// Transposed operand of a 32 x 32 square held as two blocks (columns 0..15 at
// b, 16..31 at b + 1024): lane l receives rows 16 kk + 8 (l / 32) + 0..7 of
// column l mod 32.  In a group of 16 lanes ds_read_b64_tr_b16 hands lane 4a + b
// element b of the 8-byte pieces that lanes a, a + 4, a + 8, a + 12 address:
// lane j of a group addresses row k0 + j / 4, columns c0 + 4 (j mod 4) .. + 3.
__device__ __forceinline__ f16x8 tr_run(const unsigned char* b, int kk, int lane) {
  const int grp = lane >> 4, j = lane & 15;
  const int row = 16 * kk + 8 * (grp >> 1) + (j >> 2);
  const int o = grp & 1, h = (j & 3) >> 1;
  typedef __attribute__((address_space(3))) s16x4 lds_v4;
  const unsigned char* at = b + 1024 * o + 8 * (j & 1);
  auto piece = [&](int r) __attribute__((always_inline)) {
    return (lds_v4*)(reinterpret_cast<__attribute__((address_space(3))) uint16_t*>(lds_addr(at + run_off(r, h, o))));
  };
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(piece(row));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(piece(row + 4));
  const s16x4 v[2] = {lo, hi};
  return __builtin_bit_cast(f16x8, v);
}

// what a wave computes of a stage: all its blocks, those on and below the
// diagonal, none
constexpr int kAllTag = -1, kLowerTag = -2, kIdleTag = -3;

constexpr int wait_vm(int n) { return vmcnt_only(n > 63 ? 63 : n); }
constexpr int kWaitLds = 15 | (7 << 4) | (0 << 8) | (3 << 14);     // lgkmcnt(0) only

// Row and column tile of entry l of the tiles on and below the diagonal.
__device__ __forceinline__ void triangle(int l, int& i, int& j) {
  i = static_cast<int>((sqrtf(8.0f * l + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > l) --i;
  while ((i + 1) * (i + 2) / 2 <= l) ++i;
  j = l - i * (i + 1) / 2;
}

// 8 consecutive elements of an output row from their sums of products v, in the
// output's stored scale.  a: the column operand's elements at this place (x's
// low part in kApply and kFinalLo), b: the row operand's; dpi, dq: the operands'
// diagonals at this row and these columns.
template <int MODE>
__device__ __forceinline__ void finish(float (&v)[8], const f16x8& a, const f16x8& b, float dpi, const float* dq,
                                       const OrthJob& jb) {
  if constexpr (MODE == kGram) {
    const float f = jb.so / (jb.sp * jb.sq);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
  } else if constexpr (MODE == kPoly) {
    // c R^2 + b R = c (M M + (d_i + d_j) M_ij) + b M_ij off the diagonal
    const float f = kC * jb.so / (jb.sp * jb.sq), f1 = jb.so / jb.sq;
    const float u = fmaf(kC * f1, dpi, kB * f1);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(static_cast<float>(a[e]), fmaf(kC * f1, dq[e], u), v[e] * f);
  } else if constexpr (MODE == kMul) {
    const float f = jb.so / (jb.sp * jb.sq), fp = jb.so / jb.sp, u = dpi * (jb.so / jb.sq);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = fmaf(static_cast<float>(b[e]), dq[e] * fp, fmaf(static_cast<float>(a[e]), u, v[e] * f));
  } else if constexpr (MODE == kFinal) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= 1.0f / kSQ;
  } else {
    const float d = MODE == kApply ? jb.low(dpi) : dpi;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(static_cast<float>(a[e]), d, v[e] * (1.0f / kSQ));
  }
}

// The diagonal element (at 0..7 of v) of a symmetric output: completed, then
// split into a part exact in fp16, which is returned, and the rest, left in v.
template <int MODE>
__device__ __forceinline__ float split_diagonal(float (&v)[8], int at, float dpi, float dqi, float so) {
  float d = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) d = e == at ? v[e] : d;
  if constexpr (MODE == kPoly) d = fmaf(so, fmaf(dpi, fmaf(kC, dpi, kB), kA), d);
  if constexpr (MODE == kMul) d = fmaf(so * dpi, dqi, d);
  const float e16 = static_cast<float>(static_cast<_Float16>(d));
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e == at ? d - e16 : v[e];
  return e16 / so;
}

__device__ __forceinline__ f16x8 to_f16(const float (&v)[8]) {
  f16x8 w;
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = static_cast<_Float16>(v[e]);
  return w;
}

// what rounding v to w left
__device__ __forceinline__ f16x8 low_part(const float (&v)[8], const f16x8& w) {
  f16x8 l;
#pragma unroll
  for (int e = 0; e < 8; ++e) l[e] = static_cast<_Float16>(v[e] - static_cast<float>(w[e]));
  return l;
}

__device__ __forceinline__ u32x4 to_bf16(const float (&v)[8], float f) {
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(v[2 * e] * f, v[2 * e + 1] * f);
  return o;
}

// 8 elements to (row, col) of a matrix of the caller's (any element alignment)
__device__ __forceinline__ void store_rows(bf16_t* matrix, int rows, int cols, int row, int col, const u32x4& x) {
  if (row >= rows || col >= cols) return;
  bf16_t* dst = matrix + static_cast<size_t>(row) * cols + col;
  typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
  if (col + 8 <= cols) {
    *reinterpret_cast<u32x4u*>(dst) = x;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < cols) dst[e] = static_cast<bf16_t>(x[e >> 1] >> (16 * (e & 1)));
  }
}

__device__ __forceinline__ void store_user(const OrthArgs& g, int mat, int row, int col, const u32x4& x) {
  store_rows(g.user + static_cast<size_t>(mat) * g.rows * g.cols, g.rows, g.cols, row, col, x);
}

// Halves of a lane's accumulator registers swapped with the other half wave's:
// lane l gets columns 8 (l / 32) .. + 7 of the 16 whose 8 registers c points at.
__device__ __forceinline__ void gather_columns(const float (&c)[8], float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(c[e]), __float_as_uint(c[4 + e]), false, false);
    v[e] = __uint_as_float(sw[0]);
    v[4 + e] = __uint_as_float(sw[1]);
  }
}

// One product of the iteration.  A tile is TB x TB blocks of 32 (TB = 2 WB),
// each wave owns WB x WB of them.  The symmetric modes compute the blocks on
// and below the diagonal and store the mirror image of those below.
//
// Schedule: a persistent grid walks the tiles in rounds, each round cut into 8
// runs of consecutive tiles, one per XCD (workgroup b runs on XCD b mod 8), so
// that the tiles of one matrix share an L2.  Stages go through a ring of 4; a
// stage's two MFMA steps read their operands from LDS one step ahead, one
// barrier a stage sits between them: there every wave has read the stage, so
// its buffer takes the stage four ahead (12 MFMA steps' time for the loads to
// land).  The ring runs on over tile borders.
template <int WB, int MODE>
__global__ __launch_bounds__(kOThreads, WB == 4 ? 1 : 2) void orth_gemm_kernel(OrthArgs g) {
  constexpr bool kSym = MODE <= kMul;
  constexpr bool kTr = !kSym;
  constexpr bool kOut = MODE >= kFinal;
  static_assert(WB == 2 || WB == 4, "a wave owns 2 x 2 or 4 x 4 blocks");
  constexpr int TB = 2 * WB;
  constexpr int kOpBytes = TB * 2048;               // one operand of a stage
  constexpr int kStage = 2 * kOpBytes;
  constexpr int kLoads = 2 * WB;                    // loads per wave and stage
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kStages * kStage + 4 * 4096];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave >> 1, wc = wave & 1;
  const int G = gridDim.x;
  const int mt = (g.mb + TB - 1) / TB, nt = (g.nb + TB - 1) / TB;
  const int per_mat = kSym ? mt * (mt + 1) / 2 : mt * nt;
  const int total = per_mat * g.count;
  const int nkb = g.K / kOBK;

  const int xcd = blockIdx.x % kOXcds, in_xcd = blockIdx.x / kOXcds;
  auto tile_at = [&](int r) -> int {
    const int base = r * G;
    if (base >= total) return -1;
    const int n = min(G, total - base);
    const int q = n / kOXcds, rem = n % kOXcds;
    if (in_xcd >= q + (xcd < rem ? 1 : 0)) return -1;
    return base + xcd * q + min(xcd, rem) + in_xcd;
  };

  struct Tile {
    int mat, rb, cb;                                // first row block and column block
  };
  // Sources of this wave's loads: kPtr pointers of 2 KB pieces for each
  // operand, advanced stage by stage through the tile.
  constexpr int kPtr = WB / 2;
  const unsigned char* src[2 * kPtr];
  auto locate = [&](int ti) __attribute__((always_inline)) {
    Tile t;
    t.mat = ti / per_mat;
    const int l = ti - t.mat * per_mat;
    int i, j;
    if constexpr (kSym) {
      triangle(l, i, j);
    } else {
      // column tiles vary slowly: the tiles that run together share x's columns
      j = l / mt;
      i = l - j * mt;
    }
    t.mat = __builtin_amdgcn_readfirstlane(t.mat);
    // x's row tiles are all whole: the last one starts early (its first rows
    // are written twice, with the same bits), so that every row block of a
    // wave has its stage
    t.rb = __builtin_amdgcn_readfirstlane(kTr ? min(i * TB, g.mb - TB) : i * TB);
    t.cb = __builtin_amdgcn_readfirstlane(j * TB);
    return t;
  };
  auto point = [&](const Tile& t) __attribute__((always_inline)) {
    const OrthJob& jb = g.job;
    const unsigned char* p = reinterpret_cast<const unsigned char*>(jb.p + t.mat * g.p_stride);
    const unsigned char* q = reinterpret_cast<const unsigned char*>(jb.q + t.mat * g.q_stride);
#pragma unroll
    for (int k = 0; k < kPtr; ++k) {
      // block of the operand's stage; blocks past the matrix repeat its last one
      // (in bounds, never stored)
      const int b = wave * kPtr + k;
      const int rb = min(t.rb + b, g.mb - 1), cb = min(t.cb + b, g.nb - 1);
      src[k] = uniform(p + static_cast<size_t>(rb) * (g.K >> 4) * 1024);
      src[kPtr + k] = uniform(q + (kTr ? static_cast<size_t>(2 * cb) * 1024
                                       : static_cast<size_t>(cb) * (g.K >> 4) * 1024));
    }
  };
  const uint32_t q_step = kTr ? static_cast<uint32_t>(g.nb) * 2048u : 2048u;   // bytes a stage advances q
  auto advance = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kPtr; ++k) {
      src[k] = uniform(src[k] + 2048);
      src[kPtr + k] = uniform(src[kPtr + k] + q_step);
    }
  };

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem) + wave * WB * 1024);
  const uint32_t voff[2] = {static_cast<uint32_t>(lane) * 16u, static_cast<uint32_t>(lane) * 16u + 1024u};
  // load k (0 .. 2 WB - 1) of the stage that src points at, into ring buffer buf
  auto issue = [&](int buf, int k) __attribute__((always_inline)) {
    const int o = k < WB ? 0 : 1, l = k - o * WB;   // operand, load of the operand
    const uint32_t lds = lds0 + static_cast<uint32_t>(buf * kStage + o * kOpBytes + l * 1024);
    dma_run(src[o * kPtr + l / 2], voff[l & 1], __builtin_amdgcn_readfirstlane(lds));
  };

  typedef f16x8 Frag[2 * WB];
  const uint32_t run0 = static_cast<uint32_t>(run_off(lane & 31, lane >> 5, 0));
  const uint32_t run1 = static_cast<uint32_t>(run_off(lane & 31, lane >> 5, 1));
  // operand k of a step: k < WB row block, else column block
  auto read_op = [&](int buf, int step, int k, Frag& f) __attribute__((always_inline)) {
    const unsigned char* s = smem + buf * kStage;
    if (k < WB) {
      f[k] = *reinterpret_cast<const f16x8*>(s + (2 * (wr * WB + k) + step) * 1024 + (step ? run1 : run0));
    } else if constexpr (kTr) {
      f[k] = tr_run(s + kOpBytes + (wc * WB + (k - WB)) * 2048, step, lane);
    } else {
      f[k] = *reinterpret_cast<const f16x8*>(s + kOpBytes + (2 * (wc * WB + (k - WB)) + step) * 1024 +
                                             (step ? run1 : run0));
    }
  };

  int round = 0;
  int ti = tile_at(0);
  if (ti < 0) return;
  Tile cur = locate(ti);
  point(cur);
  int ring = 0;                                     // buffer of the next stage
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) issue(s, k);
    advance();
  }
  __builtin_amdgcn_s_waitcnt(wait_vm((kStages - 1) * kLoads));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frag f0, f1;
#pragma unroll
  for (int k = 0; k < 2 * WB; ++k) read_op(0, 0, k, f0);

  while (ti >= 0) {
    f32x16 acc[WB][WB];
#pragma unroll
    for (int i = 0; i < WB; ++i)
#pragma unroll
      for (int j = 0; j < WB; ++j) acc[i][j] = f32x16{0.f};

    float dp[WB];                                   // the diagonal of the row operand at this lane's rows
#pragma unroll
    for (int i = 0; i < WB; ++i)
      dp[i] = MODE == kGram ? 0.0f
                            : g.job.dp[static_cast<size_t>(cur.mat) * g.d_stride +
                                       32 * min(cur.rb + wr * WB + i, g.mb - 1) + (lane & 31)];

    auto step = [&](const Frag& f, auto tag, auto&& op) __attribute__((always_inline)) {
      constexpr bool lower = decltype(tag)::value == kLowerTag;
#pragma unroll
      for (int i = 0; i < WB; ++i)
#pragma unroll
        for (int j = 0; j < WB; ++j) {
          if (!lower || j <= i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[WB + j], f[i], acc[i][j], 0, 0, 0);
          op(WB * i + j);
          __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr int kEvery = WB / 2;                  // one operand read (and load) per so many MFMAs

    // The diagonal's part of x <- P x: in the stage that holds the rows of row
    // block i of the wave, its accumulators also take diag(e) times those rows
    // (e is exact in fp16).
    auto diagonal = [&](int i, int st, const Frag& f) __attribute__((always_inline)) {
      f16x8 e;
      const int at = (lane & 31) - 16 * st - 8 * (lane >> 5);
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = k == at ? static_cast<_Float16>(dp[i] * kSQ) : static_cast<_Float16>(0.0f);
#pragma unroll
      for (int j = 0; j < WB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[WB + j], e, acc[i][j], 0, 0, 0);
    };
    auto stage = [&](auto tag) __attribute__((always_inline)) {
      constexpr int own = decltype(tag)::value;       // row block whose rows the stage holds, or a tag
      const int b0 = ring;
      const int b1 = (ring + 1) & (kStages - 1);
      if constexpr (own != kIdleTag) step(f0, tag, [&](int k) __attribute__((always_inline)) {
        if (k % kEvery == 0) read_op(b0, 1, k / kEvery, f1);
      });
      if constexpr (own >= 0) diagonal(own, 0, f0);
      // the next stage has landed once only the two stages issued after it
      // fly (stores of the previous tile, issued later still, only make this
      // wait longer)
      __builtin_amdgcn_s_waitcnt(wait_vm(2 * kLoads));
      __builtin_amdgcn_s_waitcnt(kWaitLds);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if constexpr (own != kIdleTag) {
        step(f1, tag, [&](int k) __attribute__((always_inline)) {
          if (k % kEvery == 0) read_op(b1, 0, k / kEvery, f0);
          if (k % kEvery == kEvery - 1) issue(b0, k / kEvery);
        });
      } else {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) issue(b0, k);
      }
      if constexpr (own >= 0) diagonal(own, 1, f1);
      advance();
      ring = b1;
    };
    // ---- what the epilogue reads beside the accumulators (block (rb, cb) of
    // the operands, diagonals) is loaded kAhead blocks ahead, the first ones
    // before the tile's last stages
    constexpr int kBlocks = WB * WB, kAhead = 4;
    const size_t o16 = static_cast<size_t>(2 * g.nb);              // 16-column blocks per output row block
    const int r = lane & 31, h = lane >> 5;
    auto row_block = [&](int i) { return cur.rb + wr * WB + i; };
    auto col_block = [&](int j) { return cur.cb + wc * WB + j; };
    // byte offset of block (rb, cb)'s 2 KB (two 16-column blocks)
    auto at_block = [&](int rb, int cb) { return (static_cast<size_t>(rb) * o16 + 2 * cb) * 1024; };
    // blocks q go down the tile's columns (kFinal: along the caller's rows)
    const bool across = kOut && !g.tall;
    struct Ahead {
      f16x8 a[2], b[MODE == kMul ? 2 : 1];
    } pre[kAhead];
    float dq[MODE == kPoly || MODE == kMul ? 2 : 1][16];
    auto run_of = [&](const _Float16* m, int64_t stride, int rb, int cb, f16x8 (&v)[2]) __attribute__((always_inline)) {
      const unsigned char* p = uniform(reinterpret_cast<const unsigned char*>(m + cur.mat * stride) + at_block(rb, cb));
      v[0] = *reinterpret_cast<const f16x8*>(p + run0);
      v[1] = *reinterpret_cast<const f16x8*>(p + 1024 + run1);
    };
    auto fetch = [&](int q) __attribute__((always_inline)) {
      if constexpr (MODE != kGram && MODE != kFinal) {
        // (blocks past the matrix: its last one, in bounds and not used)
        const int rb = min(row_block(across ? q / WB : q % WB), g.mb - 1);
        const int cb = min(col_block(across ? q % WB : q / WB), g.nb - 1);
        Ahead& e = pre[q % kAhead];
        if constexpr (MODE == kMul) run_of(g.job.p, g.p_stride, rb, cb, e.b);
        run_of(kSym ? g.job.q : g.job.lo, g.q_stride, rb, cb, e.a);
      }
    };
    auto fetch_dq = [&](int j) __attribute__((always_inline)) {
      if constexpr (MODE == kPoly || MODE == kMul) {
        const float* d = uniform(g.job.dq + static_cast<size_t>(cur.mat) * g.d_stride +
                                 32 * min(col_block(j), g.nb - 1));
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(d + 16 * p + 8 * h + 4 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) dq[j & 1][8 * p + 4 * k + e] = v[e];
          }
      }
    };
    // before the tile's last kStages stages, which load the next tile's first ones
    // (behind the last tile: this tile's again, never used, so that every wait
    // counts the same)
    const int tn = tile_at(round + 1);
    const Tile nxt = locate(max(tn, 0));
    auto turn = [&]() __attribute__((always_inline)) {
      fetch_dq(0);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) fetch(q);
      point(tn >= 0 ? nxt : cur);
    };
    using None = std::integral_constant<int, kAllTag>;
    if constexpr (kSym) {
      auto loop = [&](auto tag) __attribute__((always_inline)) {
        for (int x = kStages; x < nkb; ++x) stage(tag);
        turn();
#pragma unroll 1
        for (int x = 0; x < kStages; ++x) stage(tag);
      };
      // In a tile of R on the diagonal the blocks above it are left out (32
      // matrices of 2048 x 4096 542 -> 518 us): the upper right wave only loads,
      // the two waves on the diagonal compute their lower blocks.  The other
      // modes' epilogue loads would cross the branches, which waits for them
      // (the same matrices, Q: 314 -> 377 us).
      if (MODE != kGram || cur.rb != cur.cb || wr > wc) {
        loop(None{});
      } else if (wr == wc) {
        loop(std::integral_constant<int, kLowerTag>{});
      } else {
        loop(std::integral_constant<int, kIdleTag>{});
#pragma unroll
        for (int k = 0; k < 2 * WB; ++k) read_op(ring, 0, k, f0);
      }
    } else {
      // the stages of the wave's own row blocks apart (no branch may hold
      // MFMAs: the accumulators would leave their registers)
      int x = 0;
      auto one = [&](auto own_tag) __attribute__((always_inline)) {
        if (x == nkb - kStages) turn();
        stage(own_tag);
        ++x;
      };
      const int own = cur.rb + wr * WB;
      while (x < own) one(None{});
      one(std::integral_constant<int, 0>{});
      one(std::integral_constant<int, 1>{});
      if constexpr (WB > 2) one(std::integral_constant<int, 2>{});
      if constexpr (WB > 3) one(std::integral_constant<int, 3>{});
      while (x < nkb) one(None{});
    }

    // ---- epilogue
    const OrthJob& jb = g.job;
    unsigned char* stg = smem + kStages * kStage + wave * 4096;
    u32x4 ob[2][2];                                 // kFinal: the two blocks of a 64-element piece of rows
#pragma unroll
    for (int q = 0; q < kBlocks; ++q) {
      const int i = kOut ? q / WB : q % WB, j = kOut ? q % WB : q / WB;
      // (kFinal of a tall matrix: the same q goes down the columns)
      auto block = [&](int bi, int bj, f32x16& c) __attribute__((always_inline)) {
        // read this block's accumulators only now: without the (empty) asm the
        // compiler copies all of them out of the AGPRs at once, and spills
        if constexpr (WB == 4) asm volatile("" : "+a"(c));
        const int rb = row_block(bi), cb = col_block(bj);
        // (the other modes' fetches below must not sit in a branch)
        if (MODE == kGram && rb < cb) return;
        const bool inside = rb < g.mb && cb < g.nb;
        const bool diag = kSym && rb == cb;
        // 8 consecutive columns a lane: 16 p + 8 h + 0..7
        float v[2][8];
        const float dpi = dp[bi];
        const Ahead& pe = pre[q % kAhead];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float half[8] = {c[8 * p],     c[8 * p + 1], c[8 * p + 2], c[8 * p + 3],
                                 c[8 * p + 4], c[8 * p + 5], c[8 * p + 6], c[8 * p + 7]};
          gather_columns(half, v[p]);
          finish<MODE>(v[p], pe.a[p], pe.b[MODE == kMul ? p : 0], dpi,
                       dq[MODE == kPoly || MODE == kMul ? bj & 1 : 0] + 8 * p, jb);
        }
        if (q + kAhead < kBlocks) fetch(q + kAhead);
        f16x8 w[2], wl[2];
        if constexpr (kSym) {
          if (diag) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int at = r - 16 * p - 8 * h;    // this lane's diagonal element
              if (at >= 0 && at < 8) {
                const float dqi = MODE == kMul ? jb.dq[static_cast<size_t>(cur.mat) * g.d_stride +
                                                       32 * min(cb, g.nb - 1) + r] : 0.0f;
                const float d = split_diagonal<MODE>(v[p], at, dpi, dqi, jb.so);
                if (inside) jb.dout[static_cast<size_t>(cur.mat) * g.d_stride + 32 * rb + r] = d;
              }
            }
          }
        }
        if constexpr (!kOut) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            w[p] = to_f16(v[p]);
            if constexpr (MODE == kApply) wl[p] = low_part(v[p], w[p]);
          }
        }
        if constexpr (!kOut) {
          if (inside) {
            auto put = [&](_Float16* m, int row, int col, const f16x8 (&x)[2]) __attribute__((always_inline)) {
              unsigned char* p = uniform(reinterpret_cast<unsigned char*>(m + cur.mat * g.out_stride) + at_block(row, col));
              *reinterpret_cast<f16x8*>(p + run0) = x[0];
              *reinterpret_cast<f16x8*>(p + 1024 + run1) = x[1];
            };
            if (!kSym || rb >= cb) put(jb.out, rb, cb, w);
            if constexpr (MODE == kApply) {
              if (jb.out_lo != nullptr) put(jb.out_lo, rb, cb, wl);
            }
            if constexpr (kSym) {
              if (rb > cb) {                        // the mirror image of a block below the diagonal
                *reinterpret_cast<f16x8*>(stg + run0) = w[0];
                *reinterpret_cast<f16x8*>(stg + 1024 + run1) = w[1];
                const f16x8 t[2] = {tr_run(stg, 0, lane), tr_run(stg, 1, lane)};
                put(jb.out, cb, rb, t);
              }
            }
          }
        } else {
#pragma unroll
          for (int p = 0; p < 2; ++p) ob[q & 1][p] = to_bf16(v[p], g.scale / kSX);
        }
      };
      if constexpr (!kOut) {
        if (i == 0 && j + 1 < WB) fetch_dq(j + 1);
        block(i, j, acc[i][j]);
      } else if (!g.tall) {
        block(i, j, acc[i][j]);
      } else {
        block(j, i, acc[j][i]);
      }
      if constexpr (kOut) {
        // two blocks make 64 consecutive elements of 32 of the caller's rows:
        // through LDS (chunks XOR-swizzled by row / 2), then whole 128-byte
        // segments, 8 rows a store
        if ((q & 1) == 1) {
          if (g.tall) {
            // lane: row 32 cb + r of the caller's matrix, 8 of its columns
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              *reinterpret_cast<u32x4*>(stg + 2048 * t + run0) = ob[t][0];
              *reinterpret_cast<u32x4*>(stg + 2048 * t + 1024 + run1) = ob[t][1];
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int p = 0; p < 2; ++p) ob[t][p] = __builtin_bit_cast(u32x4, tr_run(stg + 2048 * t, p, lane));
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int p = 0; p < 2; ++p)
              *reinterpret_cast<u32x4*>(stg + r * 128 + (((4 * t + 2 * p + h) ^ ((r >> 1) & 7)) << 4)) = ob[t][p];
          // first caller row and column of the piece
          const int ur0 = 32 * (g.tall ? col_block(i) : row_block(i));
          const int uc0 = 32 * (g.tall ? row_block(j - 1) : col_block(j - 1));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 8 * k + (lane >> 3), ch = lane & 7;
            const u32x4 x = *reinterpret_cast<const u32x4*>(stg + row * 128 + ((ch ^ ((row >> 1) & 7)) << 4));
            store_user(g, cur.mat, ur0 + row, uc0 + 8 * ch, x);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    ++round;
    ti = tn;
    cur = nxt;
  }
  // trailing loads land before the workgroup's LDS is given up
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
}

// The same products for few tiles, where a tile's latency counts and not the
// matrix cores' rate: tiles of SB x SB blocks of 32, a workgroup of 8 waves
// each, which share out the stages of K.  Operands go from global memory straight into
// registers in operand order (x's blocks through 4 KB of LDS, for the
// transposing read), the loads of 2 to 8 stages a wave in flight, no barrier
// until the waves' sums are joined through LDS in a fixed order.  Wave u then
// finishes 32 rows x 16 columns, half of block u / 2.
constexpr int kSThreads = 512;
constexpr int kSWaves = kSThreads / 64;

template <int SB, int MODE>
__global__ __launch_bounds__(kSThreads) void orth_small_kernel(OrthArgs g) {
  constexpr bool kSym = MODE <= kMul;
  constexpr bool kTr = !kSym;
  constexpr bool kOut = MODE >= kFinal;
  constexpr int kHalf = kSWaves / 2;
  constexpr int kAcc = SB * SB;                       // blocks of a tile
  constexpr int kAhead = SB == 1 ? 4 : 2;             // stages a wave loads at once, two sets in turn
  // the waves' sums (half of them at a time); before that, x's blocks; behind
  // it, finished blocks on their way to a transposed store
  __shared__ __attribute__((aligned(1024))) unsigned char
      smem[(kAcc * kHalf * 4096 > kSWaves * SB * 2048 ? kAcc * kHalf * 4096 : kSWaves * SB * 2048) + kAcc * 2048];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int mt = (g.mb + SB - 1) / SB, nt = (g.nb + SB - 1) / SB;
  const int per_mat = kSym ? mt * (mt + 1) / 2 : mt * nt;
  const int total = per_mat * g.count;
  // runs of consecutive tiles on the XCDs (workgroup b runs on XCD b mod 8)
  const int per_xcd = (total + kOXcds - 1) / kOXcds;
  const int ti = (blockIdx.x % kOXcds) * per_xcd + blockIdx.x / kOXcds;
  if (ti >= total) return;
  const int mat = ti / per_mat, l = ti - mat * per_mat;
  int i0, j0;
  if constexpr (kSym) {
    triangle(l, i0, j0);
  } else {
    j0 = l / mt;
    i0 = l - j0 * mt;
  }
  // (x's row tiles are all whole, as in the kernel above)
  const int rb0 = __builtin_amdgcn_readfirstlane(kTr ? min(SB * i0, g.mb - SB) : SB * i0);
  const int cb0 = __builtin_amdgcn_readfirstlane(SB * j0);
  const OrthJob& jb = g.job;
  const unsigned char* P = reinterpret_cast<const unsigned char*>(jb.p + mat * g.p_stride);
  const unsigned char* Q = reinterpret_cast<const unsigned char*>(jb.q + mat * g.q_stride);
  const size_t row_bytes = static_cast<size_t>(g.K) * 64;      // a row block of a row-operand matrix
  const int nkb = g.K / kOBK;
  const int run[2] = {run_off(r, h, 0), run_off(r, h, 1)};
  const float* dpm = MODE == kGram ? nullptr : jb.dp + static_cast<size_t>(mat) * g.d_stride;

  f32x16 acc[SB][SB];
#pragma unroll
  for (int i = 0; i < SB; ++i)
#pragma unroll
    for (int j = 0; j < SB; ++j) acc[i][j] = f32x16{0.f};
  unsigned char* mine = smem + wave * SB * 2048;
  struct Set {
    f16x8 p[kAhead][SB][2], q[kAhead][SB][2];
  };
  auto load = [&](int base, Set& t) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      // (a stage past the end loads the last one again: in bounds, not used)
      const int kb = min(base + s * kSWaves, nkb - 1);
#pragma unroll
      for (int i = 0; i < SB; ++i) {
        const unsigned char* ps = P + min(rb0 + i, g.mb - 1) * row_bytes + kb * 2048;
        const int cb = min(cb0 + i, g.nb - 1);
        const unsigned char* qs = kTr ? Q + (static_cast<size_t>(kb) * g.nb + cb) * 2048 : Q + cb * row_bytes + kb * 2048;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          t.p[s][i][o] = *reinterpret_cast<const f16x8*>(ps + o * 1024 + run[o]);
          t.q[s][i][o] = *reinterpret_cast<const f16x8*>(qs + o * 1024 + (kTr ? lane * 16 : run[o]));
        }
      }
    }
  };
  auto use = [&](int base, Set& t) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int kb = base + s * kSWaves;
      if (kb < nkb) {
        if constexpr (kTr) {
#pragma unroll
          for (int j = 0; j < SB; ++j)
#pragma unroll
            for (int o = 0; o < 2; ++o)
              *reinterpret_cast<f16x8*>(mine + j * 2048 + o * 1024 + lane * 16) = t.q[s][j][o];
#pragma unroll
          for (int j = 0; j < SB; ++j)
#pragma unroll
            for (int st = 0; st < 2; ++st) t.q[s][j][st] = tr_run(mine + j * 2048, st, lane);
        }
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int i = 0; i < SB; ++i) {
            if constexpr (kTr) {
              // the diagonal's part: diag(e) times x's own rows
              if (kb == rb0 + i) {
                const float e16 = dpm[32 * (rb0 + i) + r] * kSQ;
                const int at = r - 16 * st - 8 * h;
                f16x8 e;
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] = k == at ? static_cast<_Float16>(e16) : static_cast<_Float16>(0.0f);
#pragma unroll
                for (int j = 0; j < SB; ++j)
                  acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(t.q[s][j][st], e, acc[i][j], 0, 0, 0);
              }
            }
#pragma unroll
            for (int j = 0; j < SB; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(t.q[s][j][st], t.p[s][i][st], acc[i][j], 0, 0, 0);
          }
      }
    }
  };
  constexpr int kStep = kSWaves * kAhead;
  Set s0, s1;
  load(wave, s0);
  for (int base = wave; base < nkb; base += 2 * kStep) {
    if (base + kStep < nkb) load(base + kStep, s1);
    use(base, s0);
    if (base + 2 * kStep < nkb) load(base + 2 * kStep, s0);
    use(base + kStep, s1);
  }

  // ---- this wave's part of the output: rows of row block i, columns 16 p .. of column block j
  const int unit = SB == 2 ? wave >> 1 : 0, p = wave & 1, ui = unit >> 1, uj = unit & 1;
  const bool finishes = wave < 2 * kAcc;                  // (of one block, two waves finish a half each)
  const int rb = rb0 + ui, cb = cb0 + uj;
  const bool inside = finishes && rb < g.mb && cb < g.nb;
  const size_t o16 = static_cast<size_t>(2 * g.nb);
  const size_t blk = ((static_cast<size_t>(min(rb, g.mb - 1)) * o16 + 2 * min(cb, g.nb - 1) + p) * 1024 + run[p]) / 2;
  f16x8 ea{}, eb{};
  float dpi = 0.0f, dq[8] = {}, dqi = 0.0f;
  if constexpr (MODE != kGram) {
    if constexpr (MODE != kFinal) ea = *reinterpret_cast<const f16x8*>((kSym ? jb.q : jb.lo) + mat * g.q_stride + blk);
    if constexpr (MODE == kMul) eb = *reinterpret_cast<const f16x8*>(jb.p + mat * g.p_stride + blk);
    dpi = dpm[32 * min(rb, g.mb - 1) + r];
  }
  if constexpr (MODE == kPoly || MODE == kMul) {
    const float* d = jb.dq + static_cast<size_t>(mat) * g.d_stride + 32 * min(cb, g.nb - 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) dq[e] = d[16 * p + 8 * h + e];
    dqi = d[r];
  }
  float* red = reinterpret_cast<float*>(smem);
  __syncthreads();                                    // x's blocks have been read
  auto exchange = [&](bool store, int slot) {
#pragma unroll
    for (int b = 0; b < kAcc; ++b)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float* at = red + ((slot * kAcc + b) * 16 + k) * 64 + lane;
        if (store) *at = acc[b / SB][b % SB][k];
        else acc[b / SB][b % SB][k] += *at;
      }
  };
  if (wave >= kHalf) exchange(true, wave - kHalf);
  __syncthreads();
  if (wave < kHalf) {
    exchange(false, wave);
    exchange(true, wave);
  }
  __syncthreads();
  float c[8], v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c[k] = 0.0f;
#pragma unroll
    for (int w = 0; w < kHalf; ++w) c[k] += red[((w * kAcc + unit) * 16 + 8 * p + k) * 64 + lane];
  }
  gather_columns(c, v);
  finish<MODE>(v, ea, eb, dpi, dq, jb);
  if constexpr (kSym) {
    const int at = r - 16 * p - 8 * h;
    if (rb == cb && at >= 0 && at < 8) {
      const float d = split_diagonal<MODE>(v, at, dpi, dqi, jb.so);
      if (inside) jb.dout[static_cast<size_t>(mat) * g.d_stride + 32 * rb + r] = d;
    }
  }
  unsigned char* flip = smem + sizeof(smem) - kAcc * 2048 + unit * 2048;
  if constexpr (!kOut) {
    const f16x8 w = to_f16(v);
    if (inside) {
      *reinterpret_cast<f16x8*>(jb.out + mat * g.out_stride + blk) = w;
      if constexpr (MODE == kApply) {
        if (jb.out_lo != nullptr) *reinterpret_cast<f16x8*>(jb.out_lo + mat * g.out_stride + blk) = low_part(v, w);
      }
    }
    if constexpr (kSym) {
      if (rb0 != cb0) {                               // the mirror image
        if (finishes) *reinterpret_cast<f16x8*>(flip + p * 1024 + run[p]) = w;
        __syncthreads();
        const f16x8 t = tr_run(flip, p, lane);
        if (inside)
          *reinterpret_cast<f16x8*>(jb.out + mat * g.out_stride +
                                    ((static_cast<size_t>(cb) * o16 + 2 * rb + p) * 1024 + run[p]) / 2) = t;
      }
    }
  } else {
    u32x4 o = to_bf16(v, g.scale / kSX);
    if (g.tall) {
      if (finishes) *reinterpret_cast<u32x4*>(flip + p * 1024 + run[p]) = o;
      __syncthreads();
      o = __builtin_bit_cast(u32x4, tr_run(flip, p, lane));
    }
    if (finishes)
      store_user(g, mat, 32 * (g.tall ? cb : rb) + r, 32 * (g.tall ? rb : cb) + 16 * p + 8 * h, o);
  }
}

// ------------------------------------------------------------------ input
constexpr int kSumThreads = 256;
// Elements per workgroup of the sums: 8 vectors a thread, fewer for small
// inputs (as long as a matrix has at most 256 partial sums).
constexpr int kSumFew = 8 * kSumThreads, kSumMany = 64 * kSumThreads;

template <typename T>
__device__ __forceinline__ float load_elem(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}

template <typename T>
__device__ __forceinline__ void store_f32x8(T* p, const float (&v)[8]) {
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[4 * k + e]);
    *reinterpret_cast<raw*>(p + 4 * k) = w;
  }
}

// 8 consecutive elements from any element's address
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
  for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k) {
    const u32x4 w = *reinterpret_cast<const raw*>(p + 4 * k);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * k + e] = __uint_as_float(w[e]);
    }
  }
}

// What u is multiplied by, in x's stored scale, from its sum of squares: an
// infinity or a NaN anywhere makes the whole matrix NaN, a zero matrix stays 0.
__device__ __forceinline__ double inverse_norm(double s, float eps) {
  const double norm = sqrt(s) + static_cast<double>(eps);
  return s < 1.0 / 0.0 ? (norm > 0.0 ? kSX / norm : 0.0) : 0.0 / 0.0;
}

// v f as ldexp(v, e) * m: in fp32, for a factor f outside its range (|v f| is
// at most kSX; m is f's mantissa rounded to fp32)
struct Factor {
  float m;
  int e;
};

__device__ __forceinline__ Factor factor_of(double f) {
  Factor r;
  r.m = static_cast<float>(frexp(f, &r.e));
  return r;
}

__device__ __forceinline__ float scaled(float v, const Factor& f) { return ldexpf(v, f.e) * f.m; }

// Sums of squares of the update u = g (or, with momentum, M <- mu M + g and
// u = g + mu M or M), 8 elements a thread at a time.  In 64 bits: bf16 values
// reach 1e38, and their squares would leave fp32.
template <typename T>
__global__ __launch_bounds__(kSumThreads) void orth_sums_kernel(const T* g, float* mom, float mu, bool nesterov,
                                                                int64_t elems, int each, int parts,
                                                                double* sums) {
  __shared__ double red[kSumThreads / 64];
  const size_t base = static_cast<size_t>(blockIdx.y) * elems;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * each;
  const int64_t end = min(first + each, elems);
  double s = 0.0;
  auto one = [&](float gv, float& m) {
    float u = gv;
    if (mom != nullptr) {
      m = fmaf(mu, m, gv);
      u = nesterov ? fmaf(mu, m, gv) : m;
    }
    s = fma(static_cast<double>(u), static_cast<double>(u), s);
  };
#pragma unroll 2
  for (int64_t i = first + 8 * threadIdx.x; i < end; i += 8 * kSumThreads) {
    float v[8], m[8];
    if (i + 8 <= end) {
      load8(g + base + i, v);
      if (mom != nullptr) load8(mom + base + i, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) one(v[e], m[e]);
      if (mom != nullptr) store_f32x8(mom + base + i, m);
    } else {
      for (int e = 0; i + e < end; ++e) {
        float x = mom != nullptr ? mom[base + i + e] : 0.0f;
        one(load_elem(g + base + i + e), x);
        if (mom != nullptr) mom[base + i + e] = x;
      }
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kSumThreads / 64; ++w) s += red[w];
    sums[static_cast<size_t>(blockIdx.y) * parts + blockIdx.x] = s;
  }
}

constexpr int kPackCols = 128;         // columns of x per workgroup (one row block)

// x_0 = u / (|u|_F + eps) as fp16 hi + lo blocks, zero outside the matrix.  The
// piece of 32 x 128 is read along the caller's rows, 8 elements a thread,
// scattered into blocks in LDS, and written as whole kilobytes.
template <typename T>
__global__ __launch_bounds__(256) void orth_pack_kernel(const T* g, const float* mom, float mu, bool nesterov,
                                                        int rows, int cols, bool tall, float eps, int parts,
                                                        const double* sums, int nb, _Float16* hi, _Float16* lo,
                                                        int64_t x_stride) {
  __shared__ __attribute__((aligned(16))) unsigned char buf[2][32 * kPackCols * 2];
  __shared__ double s_sum[4];
  const int mat = blockIdx.z, rb = blockIdx.y, c0 = blockIdx.x * kPackCols;
  const int tid = threadIdx.x;
  const size_t base = static_cast<size_t>(mat) * rows * cols;
  // unit i of 2: 8 elements along the caller's rows, from (row, col) of x
  constexpr int kUnits = 32 * kPackCols / 8 / 256;
  float u[kUnits][8];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int i = tid + 256 * k;
    const int r = tall ? 8 * (i & 3) : i / (kPackCols / 8), c = tall ? i >> 2 : 8 * (i % (kPackCols / 8));
    const int gr = 32 * rb + r, gc = c0 + c;                       // element (gr, gc) of x
    const int ur = tall ? gc : gr, uc = tall ? gr : gc;            // of the caller's matrix
    const size_t at = base + static_cast<size_t>(ur) * cols + uc;
#pragma unroll
    for (int e = 0; e < 8; ++e) u[k][e] = 0.0f;
    if (ur < rows && uc < cols) {
      float mv[8];
      if (uc + 8 <= cols) {
        load8(g + at, u[k]);
        if (mom != nullptr) load8(mom + at, mv);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[k][e] = uc + e < cols ? load_elem(g + at + e) : 0.0f;
          mv[e] = mom != nullptr && uc + e < cols ? mom[at + e] : 0.0f;
        }
      }
      if (mom != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[k][e] = nesterov ? fmaf(mu, mv[e], u[k][e]) : mv[e];
      }
    }
  }
  double s = 0.0;
  for (int i = tid; i < parts; i += 256) s += sums[static_cast<size_t>(mat) * parts + i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  if ((tid & 63) == 0) s_sum[tid >> 6] = s;
  __syncthreads();
  const Factor inv = factor_of(inverse_norm((s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]), eps));
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int i = tid + 256 * k;
    const int r = tall ? 8 * (i & 3) : i / (kPackCols / 8), c = tall ? i >> 2 : 8 * (i % (kPackCols / 8));
    f16x8 a, b;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = scaled(u[k][e], inv);
      a[e] = static_cast<_Float16>(v);
      b[e] = static_cast<_Float16>(v - static_cast<float>(a[e]));
    }
    if (!tall) {
      const int at = (c >> 4) * 1024 + run_off(r, (c >> 3) & 1, (c >> 4) & 1);
      *reinterpret_cast<f16x8*>(buf[0] + at) = a;
      *reinterpret_cast<f16x8*>(buf[1] + at) = b;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = (c >> 4) * 1024 + run_off(r + e, (c >> 3) & 1, (c >> 4) & 1) + (c & 7) * 2;
        *reinterpret_cast<_Float16*>(buf[0] + at) = a[e];
        *reinterpret_cast<_Float16*>(buf[1] + at) = b[e];
      }
    }
  }
  __syncthreads();
  const int blocks = min(kPackCols / 16, 2 * nb - c0 / 16);      // (a narrow matrix may end inside the piece)
  const size_t at = mat * x_stride + (static_cast<size_t>(rb) * 2 * nb + c0 / 16) * 512;
  for (int i = tid; i < blocks * 64; i += 256) {
    *reinterpret_cast<u32x4*>(hi + at + i * 8) = *reinterpret_cast<const u32x4*>(buf[0] + i * 16);
    *reinterpret_cast<u32x4*>(lo + at + i * 8) = *reinterpret_cast<const u32x4*>(buf[1] + i * 16);
  }
}

// ------------------------------------------------------------ small matrices
// A whole update in one workgroup, for matrices whose x fits its LDS: the
// launches of the general path would be most of the time (1 matrix of 128 x 128:
// 30 us against 58, of 128 x 400: 55 against 61; 256 of 128 x 128: 32 against
// 120, of 64 x 1000: 58 against 349).
//   * x stays in registers, in fp32 and in accumulator order: wave w owns the
//     blocks w, w + 8, ... (row block t mod MB, column block t / MB); its fp16
//     copy, the products' operand, is in LDS in blocks as above;
//   * the symmetric matrix, R and then in its place Q, is in LDS with zeros (Q:
//     what LowGain takes off the diagonal) on the diagonal and the diagonal in
//     fp32 beside it;
//   * a step: R's lower blocks dealt to the waves (for few blocks also K, the
//     parts joined through LDS in order), Q's likewise, then every wave its
//     blocks of Q x; the block's elementwise part g_i x_ij is in fp32.
constexpr int kResMaxMB = 6;
constexpr int kResBlocks = 8;                         // blocks of x a wave owns at most
constexpr int kResLoads = 4;                          // blocks whose input is loaded at once
constexpr int kResLds = 160 * 1024;

// column blocks of x that fit beside the rest
constexpr int res_split(int mb) { return mb == 1 ? 4 : mb == 2 ? 2 : 1; }
constexpr int res_fixed(int mb) {
  return mb * mb * 2048 + (res_split(mb) - 1) * (mb * (mb + 1) / 2) * 4096 + 2 * mb * 32 * 4 + 256;
}
constexpr int res_cols(int mb) {
  const int lds = (kResLds - res_fixed(mb)) / (mb * 2048), regs = kResBlocks * 8 / mb;
  return lds < regs ? lds : regs;
}

// A uniform value the compiler knows nothing about: what is computed from it
// stays where it is used (hoisted out of the steps, the addresses of every
// block would take the registers of x).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

template <typename T, int MB>
__global__ __launch_bounds__(kSThreads) void orth_resident_kernel(const T* gp, float* mom, float mu, bool nesterov,
                                                                  int rows, int cols, bool tall, int nb, int steps,
                                                                  float eps, float scale, bf16_t* out) {
  constexpr int kTri = MB * (MB + 1) / 2, kSplit = res_split(MB), kItems = kTri * kSplit;
  constexpr int kMine = (kItems + kSWaves - 1) / kSWaves;      // blocks of R a wave computes
  constexpr int kQMine = (kTri + kSWaves - 1) / kSWaves;       // blocks of Q
  constexpr int kXBytes = MB * res_cols(MB) * 2048;
  constexpr int kStageBytes = 32 * 33 * 4;                     // a block in fp32, rows padded
  static_assert(kXBytes >= kSWaves * kStageBytes, "the waves' staging blocks share x's place");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kXBytes + res_fixed(MB)];
  unsigned char* xs = smem;
  unsigned char* ms = smem + kXBytes;                          // R, then Q
  float* part = reinterpret_cast<float*>(ms + MB * MB * 2048);
  float* rd = part + (kSplit - 1) * kTri * 1024;
  float* qd = rd + 32 * MB;
  double* red = reinterpret_cast<double*>(qd + 32 * MB);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int run[2] = {run_off(r, h, 0), run_off(r, h, 1)};
  const int mat = blockIdx.x;
  const size_t base = static_cast<size_t>(mat) * rows * cols;
  const int blocks = MB * nb;
  float* stg = reinterpret_cast<float*>(xs + wave * kStageBytes);

  // ---- the update u, block by block: whole pieces of the caller's rows into
  // the wave's staging block, from there in accumulator order
  float x[kResBlocks][16];
  double ss = 0.0;
#pragma unroll
  for (int t0 = 0; t0 < kResBlocks; t0 += kResLoads) {
    float v[kResLoads][2][8], m[kResLoads][2][8];
    // half k of block t: 8 elements from (row, col) of the caller's matrix
    auto place = [&](int t, int k, int& ur, int& uc) __attribute__((always_inline)) {
      const int b = opaque(wave + kSWaves * t);
      ur = 32 * (tall ? b / MB : b % MB) + 16 * k + (lane >> 2);
      uc = 32 * (tall ? b % MB : b / MB) + 8 * (lane & 3);
      return b < blocks && ur < rows && uc < cols;
    };
#pragma unroll
    for (int s = 0; s < kResLoads; ++s)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int ur, uc;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[s][k][e] = m[s][k][e] = 0.0f;
        if (place(t0 + s, k, ur, uc)) {
          const size_t at = base + static_cast<size_t>(ur) * cols + uc;
          if (uc + 8 <= cols) {
            load8(gp + at, v[s][k]);
            if (mom != nullptr) load8(mom + at, m[s][k]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (uc + e < cols) {
                v[s][k][e] = load_elem(gp + at + e);
                if (mom != nullptr) m[s][k][e] = mom[at + e];
              }
          }
        }
      }
#pragma unroll
    for (int s = 0; s < kResLoads; ++s) {
      const int t = t0 + s;
#pragma unroll
      for (int q = 0; q < 16; ++q) x[t][q] = 0.0f;
      if (opaque(wave + kSWaves * t) >= blocks) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int ur, uc;
        const bool in = place(t, k, ur, uc);
        if (mom != nullptr) {
          // (elements past the row's end are 0 and stay 0)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            m[s][k][e] = fmaf(mu, m[s][k][e], v[s][k][e]);
            v[s][k][e] = nesterov ? fmaf(mu, m[s][k][e], v[s][k][e]) : m[s][k][e];
          }
          if (in) {
            const size_t at = base + static_cast<size_t>(ur) * cols + uc;
            if (uc + 8 <= cols) {
              store_f32x8(mom + at, m[s][k]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (uc + e < cols) mom[at + e] = m[s][k][e];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) stg[(16 * k + (lane >> 2)) * 33 + 8 * (lane & 3) + e] = v[s][k][e];
      }
      // register q of a lane: row r, column 8 (q / 4) + 4 h + q mod 4
      float big = 0.0f;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int c = 8 * (q >> 2) + 4 * h + (q & 3);
        x[t][q] = tall ? stg[c * 33 + r] : stg[r * 33 + c];
        big = fmaxf(big, fabsf(x[t][q]));
      }
      // a block's squares in fp32, relative to its largest element
      int e;
      frexpf(big, &e);
      float s2 = 0.0f;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const float y = ldexpf(x[t][q], -e);
        s2 = fmaf(y, y, s2);
      }
      ss += ldexp(static_cast<double>(s2), 2 * e);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) ss += __shfl_xor(ss, d);
  if (lane == 0) red[wave] = ss;
  __syncthreads();
  ss = 0.0;
#pragma unroll
  for (int w = 0; w < kSWaves; ++w) ss += red[w];
  const Factor inv = factor_of(inverse_norm(ss, eps));
#pragma unroll
  for (int t = 0; t < kResBlocks; ++t) {
    if (opaque(wave + kSWaves * t) >= blocks) continue;
#pragma unroll
    for (int q = 0; q < 16; ++q) x[t][q] = scaled(x[t][q], inv);
    __builtin_amdgcn_sched_barrier(0);
  }

  auto columns = [&](const float (&c)[16], int p, float (&v)[8]) __attribute__((always_inline)) {
    float half[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) half[e] = c[8 * p + e];
    gather_columns(half, v);
  };
  auto put_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < kResBlocks; ++t) {
      const int b = opaque(wave + kSWaves * t);
      if (b < blocks) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float v[8];
          columns(x[t], p, v);
          *reinterpret_cast<f16x8*>(xs + ((b % MB) * 2 * nb + 2 * (b / MB) + p) * 1024 + run[p]) = to_f16(v);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // a lower block (i, j) of the symmetric matrix and its mirror image
  auto put_sym = [&](int i, int j, const f16x8 (&w)[2]) __attribute__((always_inline)) {
    unsigned char* at = ms + (i * 2 * MB + 2 * j) * 1024;
#pragma unroll
    for (int p = 0; p < 2; ++p) *reinterpret_cast<f16x8*>(at + p * 1024 + run[p]) = w[p];
    if (i != j) {
      const f16x8 t[2] = {tr_run(at, 0, lane), tr_run(at, 1, lane)};
#pragma unroll
      for (int p = 0; p < 2; ++p)
        *reinterpret_cast<f16x8*>(ms + (j * 2 * MB + 2 * i + p) * 1024 + run[p]) = t[p];
    }
  };

  // the blocks of R and of Q this wave computes
  int gi[kMine], gj[kMine], qi[kQMine], qj[kQMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    int i, j;
    triangle((wave + kSWaves * k) / kSplit, i, j);
    gi[k] = __builtin_amdgcn_readfirstlane(i);
    gj[k] = __builtin_amdgcn_readfirstlane(j);
  }
#pragma unroll
  for (int k = 0; k < kQMine; ++k) {
    int i, j;
    triangle(wave + kSWaves * k, i, j);
    qi[k] = __builtin_amdgcn_readfirstlane(i);
    qj[k] = __builtin_amdgcn_readfirstlane(j);
  }

  for (int step = 0; step < steps; ++step) {
    put_x();
    __syncthreads();
    // ---- R = x x^T
    f32x16 acc[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      acc[k] = f32x16{0.f};
      const int it = opaque(wave + kSWaves * k);
      if (it < kItems) {
        const int i = opaque(gi[k]), j = opaque(gj[k]);
        const unsigned char* pi = xs + i * 2 * nb * 1024;
        const unsigned char* pj = xs + j * 2 * nb * 1024;
        // two stages' operands at a time
        int kb = it % kSplit;
        for (; kb + kSplit < nb; kb += 2 * kSplit) {
          f16x8 a[4], b[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int at = (2 * (kb + kSplit * (z >> 1)) + (z & 1)) * 1024 + run[z & 1];
            a[z] = *reinterpret_cast<const f16x8*>(pi + at);
            b[z] = *reinterpret_cast<const f16x8*>(pj + at);
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) acc[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[z], a[z], acc[k], 0, 0, 0);
        }
        if (kb < nb) {
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const f16x8 a = *reinterpret_cast<const f16x8*>(pi + (2 * kb + st) * 1024 + run[st]);
            const f16x8 b = *reinterpret_cast<const f16x8*>(pj + (2 * kb + st) * 1024 + run[st]);
            acc[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, a, acc[k], 0, 0, 0);
          }
        }
        if (kSplit > 1 && it % kSplit != 0) {
#pragma unroll
          for (int q = 0; q < 16; ++q)
            part[(((it % kSplit - 1) * kTri + it / kSplit) * 16 + q) * 64 + lane] = acc[k][q];
        }
      }
    }
    if constexpr (kSplit > 1) __syncthreads();
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int it = opaque(wave + kSWaves * k);
      if (it < kItems && it % kSplit == 0) {
        const int i = opaque(gi[k]), j = opaque(gj[k]);
        float c[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          c[q] = acc[k][q];
#pragma unroll
          for (int z = 0; z < kSplit - 1; ++z) c[q] += part[((z * kTri + it / kSplit) * 16 + q) * 64 + lane];
          c[q] *= 1.0f / kSX;
        }
        f16x8 w[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float v[8];
          columns(c, p, v);
          const int at = r - 16 * p - 8 * h;
          if (i == j && at >= 0 && at < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e == at) {
                rd[32 * i + r] = v[e] * (1.0f / kSX);
                v[e] = 0.0f;
              }
          }
          w[p] = to_f16(v);
        }
        put_sym(i, j, w);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    // ---- Q = a I + b R + c R^2, kept in registers until R has been read
    const LowGain low = low_gain(1, steps - 1 - step);
    f16x8 qw[kQMine][2];
#pragma unroll
    for (int k = 0; k < kQMine; ++k) {
      const int it = opaque(wave + kSWaves * k);
      if (it < kTri) {
        const int i = opaque(qi[k]), j = opaque(qj[k]);
        f32x16 a2 = f32x16{0.f};
#pragma unroll
        for (int kb = 0; kb < 2 * MB; ++kb) {
          const f16x8 a = *reinterpret_cast<const f16x8*>(ms + (i * 2 * MB + kb) * 1024 + run[kb & 1]);
          const f16x8 b = *reinterpret_cast<const f16x8*>(ms + (j * 2 * MB + kb) * 1024 + run[kb & 1]);
          a2 = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, a, a2, 0, 0, 0);
        }
        float c[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) c[q] = a2[q];
        const float di = rd[32 * i + r];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float v[8];
          columns(c, p, v);
          const f16x8 m = *reinterpret_cast<const f16x8*>(ms + (i * 2 * MB + 2 * j + p) * 1024 + run[p]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float dj = rd[32 * j + 16 * p + 8 * h + e];
            v[e] = fmaf(static_cast<float>(m[e]) * (kSQ / kSX), fmaf(kC, di + dj, kB), v[e] * (kC * kSQ / (kSX * kSX)));
          }
          const int at = r - 16 * p - 8 * h;
          if (i == j && at >= 0 && at < 8) {
            // d hi + g lo as (d - g) hi, by the product, + g x (g as rounding d - g leaves it)
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) d = e == at ? v[e] : d;
            d = fmaf(d, 1.0f / kSQ, fmaf(di, fmaf(kC, di, kB), kA));
            const float s = static_cast<float>(static_cast<_Float16>((d - low(d)) * kSQ));
            qd[32 * i + r] = fmaf(s, -1.0f / kSQ, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e == at ? s : v[e];
          }
          qw[k][p] = to_f16(v);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kQMine; ++k) {
      const int it = opaque(wave + kSWaves * k);
      if (it < kTri) {
        const int i = opaque(qi[k]), j = opaque(qj[k]);
        put_sym(i, j, qw[k]);
      }
    }
    __syncthreads();
    // ---- x <- Q x (a wave's blocks share their row, and with it Q's operands,
    // where its stride through the blocks keeps the row)
    constexpr bool kOneRow = kSWaves % MB == 0;
    f16x8 qa[2 * MB];
    auto load_q = [&](int i) __attribute__((always_inline)) {
#pragma unroll
      for (int z = 0; z < 2 * MB; ++z)
        qa[z] = *reinterpret_cast<const f16x8*>(ms + (i * 2 * MB + z) * 1024 + run[z & 1]);
    };
    if constexpr (kOneRow) load_q(wave % MB);
#pragma unroll
    for (int t = 0; t < kResBlocks; ++t) {
      const int b = opaque(wave + kSWaves * t);
      if (b < blocks) {
        const int i = b % MB, j = b / MB;
        if constexpr (!kOneRow) load_q(i);
        f32x16 y = f32x16{0.f};
#pragma unroll
        for (int kb = 0; kb < MB; ++kb)
#pragma unroll
          for (int st = 0; st < 2; ++st)
            y = __builtin_amdgcn_mfma_f32_32x32x16_f16(tr_run(xs + (kb * 2 * nb + 2 * j) * 1024, st, lane),
                                                       qa[2 * kb + st], y, 0, 0, 0);
        const float di = qd[32 * i + r];
#pragma unroll
        for (int q = 0; q < 16; ++q) x[t][q] = fmaf(di, x[t][q], y[q] * (1.0f / kSQ));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();                                           // x's copy has been read
  }

  // ---- out, through the staging blocks
#pragma unroll
  for (int t = 0; t < kResBlocks; ++t) {
    const int b = opaque(wave + kSWaves * t);
    if (b < blocks) {
      const int ib = b % MB, jb = b / MB;
      const int ur0 = 32 * (tall ? jb : ib), uc0 = 32 * (tall ? ib : jb);
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int c = 8 * (q >> 2) + 4 * h + (q & 3);
        stg[tall ? c * 33 + r : r * 33 + c] = x[t][q];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 16 * k + (lane >> 2), col = 8 * (lane & 3);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = stg[row * 33 + col + e];
        store_rows(out + base, rows, cols, ur0 + row, uc0 + col, to_bf16(v, scale / kSX));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <typename T, int MB>
void launch_resident(int64_t count, int rows, int cols, const T* g, float* mom, float mu, bool nesterov, int steps,
                     float eps, float scale, bf16_t* out, hipStream_t st) {
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  if constexpr (MB > 1) {
    if ((m + 31) / 32 < MB)
      return launch_resident<T, MB - 1>(count, rows, cols, g, mom, mu, nesterov, steps, eps, scale, out, st);
  }
  orth_resident_kernel<T, MB><<<static_cast<int>(count), kSThreads, 0, st>>>(
      g, mom, mu, nesterov, rows, cols, rows > cols, (n + 31) / 32, steps, eps, scale, out);
}

bool resident(int m, int n) {
  const int mb = (m + 31) / 32, nb = (n + 31) / 32;
  constexpr int most[kResMaxMB] = {res_cols(1), res_cols(2), res_cols(3), res_cols(4), res_cols(5), res_cols(6)};
  return mb <= kResMaxMB && nb <= most[mb - 1];
}

// -------------------------------------------------------------- workspace
struct OrthPlan {
  int m, n, mp, np, each, parts;
  size_t x_elems, s_elems;             // elements of one x and one symmetric matrix
  size_t off_x[4], off_s[4], off_d[4], off_sums, bytes;
};

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

OrthPlan plan_of(int64_t count, int rows, int cols) {
  OrthPlan p{};
  p.m = rows < cols ? rows : cols;
  p.n = rows < cols ? cols : rows;
  auto pad = [](int v) { return v <= kMinPad ? kMinPad : (v + 31) & ~31; };
  p.mp = pad(p.m);
  p.np = pad(p.n);
  const int64_t elems = static_cast<int64_t>(rows) * cols;
  p.each = kSumMany;
  if (count * elems <= int64_t{2048} * kSumFew)
    p.each = static_cast<int>((elems / 256 + kSumFew) / kSumFew) * kSumFew;
  p.parts = static_cast<int>((elems + p.each - 1) / p.each);
  p.x_elems = static_cast<size_t>(p.mp) * p.np;
  p.s_elems = static_cast<size_t>(p.mp) * p.mp;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += up256(bytes);
    return o;
  };
  for (auto& o : p.off_x) o = take(count * p.x_elems * 2);
  for (auto& o : p.off_s) o = take(count * p.s_elems * 2);
  for (auto& o : p.off_d) o = take(static_cast<size_t>(count) * p.mp * 4);
  p.off_sums = take(static_cast<size_t>(count) * p.parts * 8);
  p.bytes = at;
  return p;
}

// Whether the first two steps are taken together: a launch more, so not where
// the launches are what counts (1 matrix of 256 x 2048: 36.5 us against 34.6).
bool paired(int64_t count, int m, int n, int steps) {
  return steps >= 2 && m >= 256 && 2 * n >= 3 * m && (m >= 512 || count * m * n >= (1 << 24));
}

template <int WB, int MODE>
void launch_one(const OrthArgs& a, hipStream_t st) {
  const int slots = WB == 4 ? 256 : 512;
  const int mt = (a.mb + 2 * WB - 1) / (2 * WB), nt = (a.nb + 2 * WB - 1) / (2 * WB);
  const int64_t tiles = static_cast<int64_t>(MODE <= kMul ? mt * (mt + 1) / 2 : mt * nt) * a.count;
  const int grid = static_cast<int>(tiles < slots ? tiles : slots);
  orth_gemm_kernel<WB, MODE><<<(grid + 7) / 8 * 8, kOThreads, 0, st>>>(a);
}

template <int MODE>
void launch_mode(const OrthArgs& a, hipStream_t st) {
  auto tiles_of = [&](int blocks) {
    const int64_t mt = (a.mb + blocks - 1) / blocks, nt = (a.nb + blocks - 1) / blocks;
    return (MODE <= kMul ? mt * (mt + 1) / 2 : mt * nt) * a.count;
  };
  // One round of 32- or 64-wide tiles where they fit one (update of 1 matrix of
  // 256 x 2048: 143 us with 128-wide tiles, 122 with 64-wide ones, 99 with
  // 32-wide ones for R and Q; of 1024 x 1024: 150 with 64-wide ones, 175 with
  // 32-wide ones, two rounds); 256-wide tiles where
  // there are enough of them and K pays for their long epilogue (256 matrices
  // of 1024 x 2048: 12.1 ms against 14.5; 32 of 512 x 2048, K = 512: products
  // with x 82 us against 72 with 128-wide ones).
  if (tiles_of(1) <= 256) {
    const int64_t tiles = tiles_of(1);
    orth_small_kernel<1, MODE><<<static_cast<int>((tiles + 7) / 8 * 8), kSThreads, 0, st>>>(a);
  } else if (tiles_of(2) <= 256) {
    const int64_t tiles = tiles_of(2);
    orth_small_kernel<2, MODE><<<static_cast<int>((tiles + 7) / 8 * 8), kSThreads, 0, st>>>(a);
  } else if (tiles_of(8) >= 192 && a.mb >= 8 && (MODE <= kMul || a.K >= 1024)) {
    launch_one<4, MODE>(a, st);
  } else {
    launch_one<2, MODE>(a, st);
  }
}

}  // namespace

size_t orth_workspace_bytes(int64_t count, int rows, int cols) {
  const OrthPlan p = plan_of(count, rows, cols);
  return resident(p.m, p.n) ? 256 : p.bytes;
}

hipError_t launch_orthogonalize(int64_t count, int rows, int cols, bool bf16, const void* g, float* mom, float mu,
                                bool nesterov, int steps, float eps, float scale, bf16_t* out, void* workspace,
                                hipStream_t st) {
  const OrthPlan p = plan_of(count, rows, cols);
  if (resident(p.m, p.n)) {
    if (bf16)
      launch_resident<bf16_t, kResMaxMB>(count, rows, cols, static_cast<const bf16_t*>(g), mom, mu, nesterov, steps,
                                         eps, scale, out, st);
    else
      launch_resident<float, kResMaxMB>(count, rows, cols, static_cast<const float*>(g), mom, mu, nesterov, steps,
                                        eps, scale, out, st);
    return hipGetLastError();
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  _Float16* X[4];
  _Float16* S[4];
  float* D[4];
  for (int i = 0; i < 4; ++i) X[i] = reinterpret_cast<_Float16*>(ws + p.off_x[i]);
  for (int i = 0; i < 4; ++i) S[i] = reinterpret_cast<_Float16*>(ws + p.off_s[i]);
  for (int i = 0; i < 4; ++i) D[i] = reinterpret_cast<float*>(ws + p.off_d[i]);
  double* sums = reinterpret_cast<double*>(ws + p.off_sums);
  const bool tall = rows > cols;
  const int64_t elems = static_cast<int64_t>(rows) * cols;
  const int n = static_cast<int>(count);
  const dim3 gs(p.parts, n), gp((p.np + kPackCols - 1) / kPackCols, p.mp / 32, n);
  if (bf16) {
    const bf16_t* gb = static_cast<const bf16_t*>(g);
    orth_sums_kernel<bf16_t><<<gs, kSumThreads, 0, st>>>(gb, mom, mu, nesterov, elems, p.each, p.parts, sums);
    orth_pack_kernel<bf16_t><<<gp, 256, 0, st>>>(gb, mom, mu, nesterov, rows, cols, tall, eps, p.parts, sums,
                                                 p.np / 32, X[0], X[1], p.x_elems);
  } else {
    const float* gf = static_cast<const float*>(g);
    orth_sums_kernel<float><<<gs, kSumThreads, 0, st>>>(gf, mom, mu, nesterov, elems, p.each, p.parts, sums);
    orth_pack_kernel<float><<<gp, 256, 0, st>>>(gf, mom, mu, nesterov, rows, cols, tall, eps, p.parts, sums,
                                                p.np / 32, X[0], X[1], p.x_elems);
  }

  OrthArgs base{};
  base.count = n;
  base.mb = p.mp / 32;
  base.d_stride = p.mp;
  base.rows = rows;
  base.cols = cols;
  base.tall = tall;
  base.scale = scale;
  base.user = out;
  const int64_t xs = static_cast<int64_t>(p.x_elems), ss = static_cast<int64_t>(p.s_elems);
  int xi = 0;                                   // x lives in X[xi], X[xi + 1]
  enum { R = 0, T = 1, U = 2, V = 3 };
  auto sym_args = [&] {
    OrthArgs a = base;
    a.nb = p.mp / 32;
    a.K = p.mp;
    a.p_stride = a.q_stride = a.out_stride = ss;
    return a;
  };
  auto gram = [&] {
    OrthArgs a = sym_args();
    a.K = p.np;
    a.p_stride = a.q_stride = xs;
    a.job = {X[xi], X[xi], nullptr, nullptr, nullptr, S[R], nullptr, D[R], kSX, kSX, kSX};
    launch_mode<kGram>(a, st);
  };
  auto poly = [&](int q) {                      // S[q] = Q(S[R])
    OrthArgs a = sym_args();
    a.job = {S[R], S[R], nullptr, D[R], D[R], S[q], nullptr, D[q], kSX, kSX, kSQ};
    launch_mode<kPoly>(a, st);
  };
  auto product = [&](int pm, float sp, int qm, float sq, int om, float so) -> OrthJob {
    return {S[pm], S[qm], nullptr, D[pm], D[qm], S[om], nullptr, D[om], sp, sq, so};
  };
  auto mul = [&](const OrthJob& j) {
    OrthArgs a = sym_args();
    a.job = j;
    launch_mode<kMul>(a, st);
  };
  bool has_lo = true;                           // x_0 has a low part
  // x <- S[q] x, the polynomials of `taken` steps, with `after` steps to follow
  auto apply = [&](int q, int taken, int after) {
    OrthArgs a = base;
    a.nb = p.np / 32;
    a.K = p.mp;
    a.p_stride = ss;
    a.q_stride = a.out_stride = xs;
    a.job = {S[q], X[xi], X[xi + 1], D[q], nullptr, X[xi ^ 2], after > 1 ? X[(xi ^ 2) + 1] : nullptr, nullptr, kSQ, kSX, kSX,
             low_gain(taken, after)};
    if (after > 0) launch_mode<kApply>(a, st);
    else if (has_lo) launch_mode<kFinalLo>(a, st);
    else launch_mode<kFinal>(a, st);
    has_lo = after > 1;
    xi ^= 2;
  };

  int left = steps;
  if (paired(count, p.m, p.n, steps)) {
    gram();
    poly(U);                                    // Q1
    mul(product(U, kSQ, R, kSX, T, kSX));       // T = Q1 R
    mul(product(T, kSX, U, kSQ, R, kSX));       // R' = T Q1
    poly(V);                                    // Q2
    mul(product(V, kSQ, U, kSQ, T, kSQ));       // Q2 Q1
    left -= 2;
    apply(T, 2, left);
  }
  while (left > 0) {
    gram();
    poly(U);
    apply(U, 1, --left);
  }
  return hipGetLastError();
}

}  // namespace moe
