// The block's pre-norm and its backward pass: RMS norm ("Laguna-M.1-base",
// Normalisation: RMS norm, computed in fp32) and layer norm, with the residual
// addition in front of it.
//
// Forward, per row of width D:
//   s = x + r (rounded to elem; s = x without a residual)
//   mean = sum s / D (layer norm; 0 for RMS), rstd = 1 / sqrt(sum (s - mean)^2 / D + eps)
//   y = (s - mean) rstd gamma + beta
// Backward, with h = (s - mean) rstd and t = dy gamma:
//   ds = rstd (t - h sum(t h) / D - sum t / D [layer norm only]) + dsum
//   dgamma = sum over rows of dy h,  dbeta = sum over rows of dy
//
// Both are bound by HBM: each input is read once and each output written once
// (of few rows, the backward pass reads x and dy a second time, for the columns).
//   * A row lives in the registers of a group of 16 to 1024 threads, CH 16-byte
//     vectors a thread, so the variance is summed around the mean (no
//     cancellation) without a second read.  Past 8192 columns the backward pass
//     with column sums needs more than the 128 registers a thread of 1024 has,
//     and spills: 36 bytes a thread in bf16 (dbeta too: 108), 108 in fp32 (184).
//     4096 x 16384 with dsum, bf16: 102 us without sums (5.3 TB/s), 113 with
//     dgamma's (4.7), 148 with both (3.6); fp32: 211, 222 and 261 (4.1).
//   * Groups walk the rows with the grid as stride; gamma and beta stay in
//     registers, and in the backward pass so do the column sums of dgamma and
//     dbeta.  Each workgroup writes its sums once, to the workspace, and a
//     second kernel adds them in a fixed order: no atomics, the same bits on
//     every call.  Of few rows, workgroups of their own sum the columns in the
//     same launch (dgamma and dbeta need no sum over a row).
//   * Rows of any width: the vectors are loaded from wherever the row starts
//     (global loads take any element alignment); a last vector that is not
//     whole is cut out of the one that ends with the row.
// Sums, statistics and weight gradients are fp32.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct Vec;
template <>
struct Vec<bf16_t> {
  static constexpr int kN = 8;
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4)));
};

// the vector of a row that starts at element c (c < cols), as it is stored;
// elements past the row's end are 0.  A ragged last vector comes out of the one
// that ends with the row, shifted (element by element: 32768 x 100 in bf16, the
// backward pass, 26.8 us instead of 19.9).
template <typename T>
__device__ __forceinline__ u32x4 load_raw(const T* row, int c, int cols) {
  constexpr int N = Vec<T>::kN;
  typedef typename Vec<T>::raw raw;
  if (c + N <= cols) return *reinterpret_cast<const raw*>(row + c);
  u32x4 w = {0, 0, 0, 0};
  if (cols >= N) {
    w = *reinterpret_cast<const raw*>(row + cols - N);
    const int s = c + N - cols;                       // elements to drop
    const int words = N == 8 ? s >> 1 : s;
    if (words & 1) w = u32x4{w[1], w[2], w[3], 0};
    if (words & 2) w = u32x4{w[2], w[3], 0, 0};
    if (N == 8 && (s & 1))
      w = u32x4{(w[0] >> 16) | (w[1] << 16), (w[1] >> 16) | (w[2] << 16), (w[2] >> 16) | (w[3] << 16), w[3] >> 16};
    return w;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (c + i < cols) {
      if constexpr (N == 8) w[i >> 1] |= static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
      else w[i] = __float_as_uint(row[c + i]);
    }
  return w;
}

template <int N>
__device__ __forceinline__ void unpack(const u32x4& w, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (N == 8) v[i] = __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    else v[i] = __uint_as_float(w[i]);
  }
}

template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int c, int cols, float (&v)[Vec<T>::kN]) {
  unpack(load_raw(row, c, cols), v);
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int c, int cols, const float (&v)[Vec<T>::kN]) {
  constexpr int N = Vec<T>::kN;
  if (c + N <= cols) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 8) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      else w[i] = __float_as_uint(v[i]);
    }
    *reinterpret_cast<typename Vec<T>::raw*>(row + c) = w;
  } else {
    // pieces of 4, 2 and 1 elements
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 8) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      else w[i] = __float_as_uint(v[i]);
    }
    const int n = cols - c;
    T* p = row + c;
    typedef uint32_t two __attribute__((ext_vector_type(2), aligned(2)));
    typedef uint32_t one __attribute__((aligned(2)));
    if constexpr (N == 8) {
      if (n & 4) {
        *reinterpret_cast<two*>(p) = two{w[0], w[1]};
        p += 4;
        w = u32x4{w[2], w[3], 0, 0};
      }
      if (n & 2) {
        *reinterpret_cast<one*>(p) = w[0];
        p += 2;
        w[0] = w[1];
      }
      if (n & 1) *p = static_cast<T>(w[0]);
    } else {
      if (n & 2) {
        *reinterpret_cast<two*>(p) = two{w[0], w[1]};
        p += 2;
        w[0] = w[2];
      }
      if (n & 1) *p = __uint_as_float(w[0]);
    }
  }
}

// N elements of an fp32 row vector of the weight's length; null: `fill`
template <int N>
__device__ __forceinline__ void load_weight(const float* w, int c, int cols, float fill, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = fill;
  if (w == nullptr || c >= cols) return;
  if (c + N <= cols) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const f32x4 q = *reinterpret_cast<const f32x4u*>(w + c + 4 * k);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * k + i] = q[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < cols) v[i] = w[c + i];
  }
}

// sums of K values over the TPR threads of a row's group; every thread gets them
template <int TPR, int K>
__device__ __forceinline__ void group_sum(float (&s)[K], float* red) {
#pragma unroll
  for (int d = (TPR < 64 ? TPR : 64) / 2; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += __shfl_xor(s[k], d);
  if constexpr (TPR > 64) {
    constexpr int WPR = TPR / 64;
    // (the barriers are the workgroup's: its groups take them together)
    const int w = (threadIdx.x >> 6) % WPR;
    red += (threadIdx.x >> 6) / WPR * K * WPR;
    __syncthreads();                                  // the last call's reads are done
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[k * WPR + w] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) t += red[k * WPR + i];
      s[k] = t;
    }
  }
}

// rows at a time per workgroup
constexpr int groups_of(int tpr, bool backward) { return tpr <= 64 ? 256 / tpr : tpr == 256 && backward ? 2 : 1; }
constexpr int threads_of(int tpr, bool backward) { return tpr * groups_of(tpr, backward); }

struct NormArgs {
  const void* x;
  const void* residual;      // forward: r; backward: dsum
  const void* dy;
  const float* gamma;
  const float* beta;
  float* mean;               // forward: out, backward: in
  float* rstd;
  void* sum;
  void* y;                   // forward: y; backward: dx
  float* part;               // backward: [workgroups][2][cols] (or [1] without dbeta)
  float* dgamma;             // kOwnSums
  float* dbeta;
  int row_blocks;            // backward: workgroups that walk the rows
  int64_t rows;
  int cols;
  int layer;
  float eps;
};

template <typename T, int CH, int TPR>
__global__ __launch_bounds__(threads_of(TPR, false)) void norm_forward_kernel(NormArgs a) {
  constexpr int N = Vec<T>::kN, kT = TPR, kG = groups_of(TPR, false);
  static_assert(TPR <= 64 || kG == 1, "the groups of a workgroup would part at a barrier");
  __shared__ float red[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % kT, grp = threadIdx.x / kT;
  const int cols = a.cols;
  const float inv = 1.0f / static_cast<float>(cols);
  float gm[CH][N], bt[CH][N];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (k * kT + t) * N;
    load_weight<N>(a.gamma, c, cols, 1.0f, gm[k]);
    load_weight<N>(a.beta, c, cols, 0.0f, bt[k]);
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kG + grp; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kG) {
    const size_t at = static_cast<size_t>(row) * cols;
    float v[CH][N];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * kT + t) * N;
      if (c < cols) {
        load_vec<T>(static_cast<const T*>(a.x) + at, c, cols, v[k]);
        if (a.residual != nullptr) {
          float r[N];
          load_vec<T>(static_cast<const T*>(a.residual) + at, c, cols, r);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            v[k][i] += r[i];
            // the norm reads the sum as it is stored, as the backward pass will
            if constexpr (N == 8) v[k][i] = bf16_to_f32(f32_to_bf16(v[k][i]));
          }
          store_vec<T>(static_cast<T*>(a.sum) + at, c, cols, v[k]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[k][i] = 0.0f;
      }
    }
    float mean = 0.0f;
    if (a.layer) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += v[k][i];
      group_sum<TPR, 1>(s, red);
      mean = s[0] * inv;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if ((k * kT + t) * N + i < cols) {
          v[k][i] -= mean;
          q[0] = fmaf(v[k][i], v[k][i], q[0]);
        }
      }
    group_sum<TPR, 1>(q, red);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv, a.eps));
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * kT + t) * N;
      if (c < cols) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[k][i] = fmaf(v[k][i] * rstd, gm[k][i], bt[k][i]);
        store_vec<T>(static_cast<T*>(a.y) + at, c, cols, v[k]);
      }
    }
  }
}

// What a backward launch does beside dx: the column sums of dgamma, of dgamma
// and dbeta, or all of both by workgroups of their own.
enum { kSumGamma = 0, kSumBoth = 1, kOwnSums = 2 };

template <typename T>
__device__ __forceinline__ float elem(const void* p, size_t i) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(static_cast<const T*>(p)[i]);
  else return static_cast<const T*>(p)[i];
}

// dgamma and dbeta of THREADS / 32 columns: 32 slices of the rows, then the
// slices, both in a fixed order.
template <typename T, int THREADS>
__device__ __forceinline__ void column_sums(const NormArgs& a, int block) {
  constexpr int kSlices = 32, kCols = THREADS / kSlices;
  __shared__ float red[2][THREADS];
  const int c = block * kCols + threadIdx.x % kCols, sl = threadIdx.x / kCols;
  float g = 0.0f, b = 0.0f;
  if (c < a.cols) {
#pragma unroll 8
    for (int r = sl; r < static_cast<int>(a.rows); r += kSlices) {
      const size_t at = static_cast<size_t>(r) * a.cols + c;
      const float dy = elem<T>(a.dy, at), x = elem<T>(a.x, at);
      g = fmaf(dy, (x - (a.layer ? a.mean[r] : 0.0f)) * a.rstd[r], g);
      b += dy;
    }
  }
  red[0][threadIdx.x] = g;
  red[1][threadIdx.x] = b;
  __syncthreads();
  if (sl < 2 && c < a.cols) {                       // the first slice joins dgamma, the second dbeta
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) s += red[sl][i * kCols + threadIdx.x % kCols];
    float* out = sl ? a.dbeta : a.dgamma;
    if (out != nullptr) out[c] = s;
  }
}

template <typename T, int CH, int TPR, int SUMS>
__global__ __launch_bounds__(threads_of(TPR, true)) void norm_backward_kernel(NormArgs a) {
  constexpr bool BETA = SUMS == kSumBoth;
  if constexpr (SUMS == kOwnSums) {
    if (static_cast<int>(blockIdx.x) >= a.row_blocks)
      return column_sums<T, threads_of(TPR, true)>(a, blockIdx.x - a.row_blocks);
  }
  constexpr int N = Vec<T>::kN, kT = TPR, kG = groups_of(TPR, true);
  __shared__ float red[TPR > 64 ? 2 * TPR / 64 * kG : 1];
  __shared__ float fold[kG > 1 ? (kG - 1) * kT * N : 1];
  const int t = threadIdx.x % kT, grp = threadIdx.x / kT;
  const int cols = a.cols;
  const float inv = 1.0f / static_cast<float>(cols);
  float gm[CH][N], dg[CH][N], db[BETA ? CH : 1][N];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    load_weight<N>(a.gamma, (k * kT + t) * N, cols, 1.0f, gm[k]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dg[k][i] = 0.0f;
      if constexpr (BETA) db[k][i] = 0.0f;
    }
  }
  // a row's input, loaded while the row before it is worked on
  struct Row {
    u32x4 x[CH], dy[CH], ds[CH];
    float mean, rstd;
  } cur, next;
  auto load = [&](int64_t row0, Row& q) __attribute__((always_inline)) {
    // (a group past the last row goes through the barriers with zeros)
    const bool live = row0 + grp < a.rows;
    const int64_t row = live ? row0 + grp : a.rows - 1;
    const size_t at = static_cast<size_t>(row) * cols;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * kT + t) * N;
      q.x[k] = q.dy[k] = q.ds[k] = u32x4{0, 0, 0, 0};
      if (live && c < cols) {
        q.x[k] = load_raw(static_cast<const T*>(a.x) + at, c, cols);
        q.dy[k] = load_raw(static_cast<const T*>(a.dy) + at, c, cols);
        if (a.residual != nullptr) q.ds[k] = load_raw(static_cast<const T*>(a.residual) + at, c, cols);
      }
    }
    q.mean = a.layer ? a.mean[row] : 0.0f;
    q.rstd = a.rstd[row];
  };
  // (the widest rows leave no registers for it)
  constexpr bool kEarly = TPR < 1024 || CH == 1;
  const int64_t stride = static_cast<int64_t>(a.row_blocks) * kG;
  if (kEarly) load(static_cast<int64_t>(blockIdx.x) * kG, cur);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kG; row0 < a.rows; row0 += stride) {
    // (dx may be dy, x or dsum itself: other rows than those still to be read)
    if (!kEarly) load(row0, cur);
    else if (row0 + stride < a.rows) load(row0 + stride, next);
    float h[CH][N], g[CH][N];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      unpack(cur.x[k], h[k]);
      unpack(cur.dy[k], g[k]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // (past the row's end g is 0, so h adds nothing there)
        h[k][i] = (h[k][i] - cur.mean) * cur.rstd;
        if constexpr (SUMS != kOwnSums) dg[k][i] = fmaf(g[k][i], h[k][i], dg[k][i]);
        if constexpr (BETA) db[k][i] += g[k][i];
        g[k][i] *= gm[k][i];
        s[0] = fmaf(g[k][i], h[k][i], s[0]);
        s[1] += g[k][i];
      }
    }
    group_sum<TPR, 2>(s, red);
    const float mh = s[0] * inv, m1 = a.layer ? s[1] * inv : 0.0f;
    if (row0 + grp < a.rows) {
      T* dx = static_cast<T*>(a.y) + static_cast<size_t>(row0 + grp) * cols;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = (k * kT + t) * N;
        if (c < cols) {
          float r[N];
          unpack(cur.ds[k], r);
#pragma unroll
          for (int i = 0; i < N; ++i) r[i] = fmaf(cur.rstd, g[k][i] - m1 - h[k][i] * mh, r[i]);
          store_vec<T>(dx, c, cols, r);
        }
      }
    }
    if (kEarly) cur = next;
  }
  if (SUMS == kOwnSums || a.part == nullptr) return;
  // the workgroup's column sums: its groups' added in order, then stored
  float* part = a.part + static_cast<size_t>(blockIdx.x) * (BETA ? 2 : 1) * cols;
#pragma unroll
  for (int b = 0; b < (BETA ? 2 : 1); ++b)
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if constexpr (BETA) v[i] = b ? db[k][i] : dg[k][i];
        else v[i] = dg[k][i];
      }
      if constexpr (kG > 1) {
        __syncthreads();
        if (grp > 0) {
#pragma unroll
          for (int i = 0; i < N; ++i) fold[((grp - 1) * N + i) * kT + t] = v[i];
        }
        __syncthreads();
        if (grp == 0) {
#pragma unroll
          for (int q = 0; q < kG - 1; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += fold[(q * N + i) * kT + t];
        }
      }
      const int c = (k * kT + t) * N;
      if (grp == 0) {
        float* p = part + static_cast<size_t>(b) * cols + c;
        if (c + N <= cols) {
#pragma unroll
          for (int i = 0; i < N; i += 4) *reinterpret_cast<f32x4u*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (c + i < cols) p[i] = v[i];
        }
      }
    }
}

// out[c] = sum over workgroups of part[w][b][c]: slices of the workgroups
// for each of COLS columns, then the slices, both in a fixed order.  Bound by
// latency: every thread's loads are in flight together.
constexpr int kFoldThreads = 1024;

template <int COLS>
__global__ __launch_bounds__(kFoldThreads) void norm_fold_kernel(const float* part, int groups, int nb, int cols,
                                                                 float* dgamma, float* dbeta) {
  constexpr int kSlices = kFoldThreads / COLS;
  __shared__ float red[kFoldThreads];
  const int c = blockIdx.x * COLS + threadIdx.x % COLS, sl = threadIdx.x / COLS;
  const int b = blockIdx.y;
  float* out = b ? dbeta : dgamma;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int w = sl; w < groups; w += kSlices) s += part[(static_cast<size_t>(w) * nb + b) * cols + c];
  }
  red[threadIdx.x] = s;
#pragma unroll
  for (int n = kSlices; n > 1;) {
    // (four at a time; a last pair alone)
    const int each = n >= 4 ? 4 : 2;
    n /= each;
    __syncthreads();
    if (sl < n) {
      s = red[threadIdx.x] + red[threadIdx.x + n * COLS];
      if (each == 4) s += red[threadIdx.x + 2 * n * COLS] + red[threadIdx.x + 3 * n * COLS];
    }
    __syncthreads();
    if (sl < n) red[threadIdx.x] = s;
  }
  if (sl == 0 && c < cols && out != nullptr) out[c] = s;
}

// Vectors per thread (ch) and threads per row (tpr).  Narrow rows share a wave
// (32768 x 64 in bf16, forward: 6.7 us with 16 threads a row, 16.6 with 64).
// Batches of many rows take the fewest waves whose registers leave enough
// of them resident (32768 x 2048 in bf16, forward: 99 us with one vector and 256
// threads, 124 us with four vectors and 64; 8000 x 4097: 65 us with three and
// 256, 84 us with one and 1024); few rows are spread over more waves, for
// latency.
constexpr int kManyRows = 1024;

struct NormForm {
  int ch, tpr;
};

NormForm form_of(int64_t rows, int cols, int n) {
  const int vecs = (cols + n - 1) / n;
  auto fits = [&](int ch, int tpr) { return vecs <= ch * tpr; };
  const bool many = rows >= kManyRows;
  for (int tpr = 16; tpr <= 64; tpr *= 2)
    if (fits(1, tpr)) return {1, tpr};
  if (many && fits(2, 64)) return {2, 64};
  for (int ch = 1; ch <= (many ? 3 : 1); ++ch)
    if (fits(ch, 256)) return {ch, 256};
  for (int ch = 1; ch <= 4; ch *= 2)
    if (fits(ch, 1024)) return {ch, 1024};
  return {0, 0};
}

// Workgroups: at most what the CUs hold at once by the kernels' registers.  A
// backward pass of few rounds takes one a CU, for fewer partial sums (2048 x 2048
// in bf16: 13.3 us instead of 15.2 with two).  Grows with the rows.
int64_t most_of(int64_t rows, NormForm f, bool backward) {
  const int64_t need = (rows + groups_of(f.tpr, backward) - 1) / groups_of(f.tpr, backward);
  int per_cu = f.tpr == 1024 ? 1 : f.ch == 1 ? 6 : f.ch == 2 ? 4 : 3;
  if (backward) {
    if (f.tpr == 256) per_cu = f.ch == 1 ? 2 : 1;
    else if (f.tpr == 64) per_cu = f.ch == 1 ? 4 : 3;
    else if (f.tpr < 64) per_cu = 2;
    if (need <= 4 * 256) per_cu = 1;
  }
  const int64_t most = 256 * per_cu;
  return need < most ? need : most;
}

// The same number of rows for each workgroup (2048 workgroups instead of 1536 for
// 32768 x 2048, forward, a second round for some: 124 us instead of 99).
int grid_of(int64_t rows, NormForm f, bool backward) {
  const int64_t need = (rows + groups_of(f.tpr, backward) - 1) / groups_of(f.tpr, backward);
  const int64_t most = most_of(rows, f, backward);
  const int64_t each = (need + most - 1) / most;
  return static_cast<int>((need + each - 1) / each);
}

template <typename T, int CH, int TPR>
void launch_fwd(const NormArgs& a, int grid, hipStream_t st) {
  norm_forward_kernel<T, CH, TPR><<<grid, threads_of(TPR, false), 0, st>>>(a);
}

template <typename T, int CH, int TPR>
void launch_bwd(const NormArgs& a, int sums, hipStream_t st) {
  constexpr int kThreads = threads_of(TPR, true);
  // (few rows: one of the forms that form_of gives them)
  if constexpr (CH == 1 || TPR == 1024) {
    if (sums == kOwnSums) {
      norm_backward_kernel<T, CH, TPR, kOwnSums><<<a.row_blocks + (a.cols + kThreads / 32 - 1) / (kThreads / 32),
                                                   kThreads, 0, st>>>(a);
      return;
    }
  }
  if (sums == kSumBoth) norm_backward_kernel<T, CH, TPR, kSumBoth><<<a.row_blocks, kThreads, 0, st>>>(a);
  else norm_backward_kernel<T, CH, TPR, kSumGamma><<<a.row_blocks, kThreads, 0, st>>>(a);
}

template <typename T, typename F>
void with_form(NormForm f, F&& go) {
#define MOE_NORM_CASE(CH, TPR) \
  if (f.ch == CH && f.tpr == TPR) return go(std::integral_constant<int, CH>{}, std::integral_constant<int, TPR>{});
  MOE_NORM_CASE(1, 16) MOE_NORM_CASE(1, 32)
  MOE_NORM_CASE(1, 64) MOE_NORM_CASE(2, 64)
  MOE_NORM_CASE(1, 256) MOE_NORM_CASE(2, 256) MOE_NORM_CASE(3, 256)
  MOE_NORM_CASE(1, 1024) MOE_NORM_CASE(2, 1024)
  if constexpr (sizeof(T) == 4) { MOE_NORM_CASE(4, 1024) }
#undef MOE_NORM_CASE
}

}  // namespace

size_t norm_workspace_bytes(int64_t rows, int cols) {
  // the most workgroups of any form of this many rows or fewer, two sums each: a
  // batch's workspace also serves smaller ones
  int64_t most = 0;
  for (int n = 4; n <= 8; n += 4)
    for (int64_t r : {rows < kManyRows ? rows : int64_t{kManyRows - 1}, rows}) {
      const int64_t groups = most_of(r, form_of(r, cols, n), true);
      most = groups > most ? groups : most;
    }
  return (static_cast<size_t>(most) * 2 * cols * sizeof(float) + 255) & ~static_cast<size_t>(255);
}

hipError_t launch_norm_forward(bool layer, int64_t rows, int cols, bool bf16, const void* x, const void* residual,
                               const float* gamma, const float* beta, float eps, void* sum, void* y, float* mean,
                               float* rstd, hipStream_t st) {
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.beta = beta;
  a.mean = mean;
  a.rstd = rstd;
  a.sum = sum;
  a.y = y;
  a.rows = rows;
  a.cols = cols;
  a.layer = layer;
  a.eps = eps;
  const NormForm f = form_of(rows, cols, bf16 ? 8 : 4);
  const int grid = grid_of(rows, f, false);
  if (bf16) with_form<bf16_t>(f, [&](auto ch, auto w) { launch_fwd<bf16_t, ch(), w()>(a, grid, st); });
  else with_form<float>(f, [&](auto ch, auto w) { launch_fwd<float, ch(), w()>(a, grid, st); });
  return hipGetLastError();
}

hipError_t launch_norm_backward(bool layer, int64_t rows, int cols, bool bf16, const void* dy, const void* x,
                                const float* gamma, const float* mean, const float* rstd, const void* dsum,
                                void* dx, float* dgamma, float* dbeta, void* workspace, hipStream_t st) {
  NormArgs a{};
  a.x = x;
  a.residual = dsum;
  a.dy = dy;
  a.gamma = gamma;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.y = dx;
  a.rows = rows;
  a.cols = cols;
  a.layer = layer;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  const bool any = dgamma != nullptr || dbeta != nullptr, beta = dbeta != nullptr;
  // Few rows: dgamma and dbeta by workgroups of their own in the same launch,
  // which read x and dy once more (out of the caches) instead of writing and
  // joining partial sums: 777 x 1023 in fp32 7.3 us instead of 9.7, 64 x 4096 in
  // bf16 3.9 instead of 7.7, 1000 x 2048 11.5 against 11.2, 2500 x 2048 23.3
  // against 16.0.  Not where dx overwrites what they read.
  const bool own = any && rows > 0 && rows < kManyRows && dx != dy && dx != x;
  a.part = any ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    const NormForm f = form_of(rows, cols, bf16 ? 8 : 4);
    a.row_blocks = grid_of(rows, f, true);
    const int sums = own ? kOwnSums : beta ? kSumBoth : kSumGamma;
    if (bf16) with_form<bf16_t>(f, [&](auto ch, auto w) { launch_bwd<bf16_t, ch(), w()>(a, sums, st); });
    else with_form<float>(f, [&](auto ch, auto w) { launch_bwd<float, ch(), w()>(a, sums, st); });
  }
  if (any && !own) {
    auto fold = [&](auto c) {
      constexpr int kCols = decltype(c)::value;
      norm_fold_kernel<kCols><<<dim3((cols + kCols - 1) / kCols, beta ? 2 : 1), kFoldThreads, 0, st>>>(
          static_cast<const float*>(workspace), a.row_blocks, beta ? 2 : 1, cols, dgamma, dbeta);
    };
    // (wide rows: whole 128-byte lines; 4096 x 8192 in bf16 61.8 -> 59.0 us, 4000
    // x 64 8.4 -> 9.3 us)
    if (cols > 1024) fold(std::integral_constant<int, 32>{});
    else fold(std::integral_constant<int, 16>{});
  }
  return hipGetLastError();
}

}  // namespace moe
