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
// Both are bound by HBM: each input is read once and each output written once.
//   * A row lives in the registers of a group of 1, 4 or 16 waves, CH 16-byte
//     vectors a thread, so the variance is summed around the mean (no
//     cancellation) without a second read.
//   * Groups walk the rows with the grid as stride; gamma and beta stay in
//     registers, and in the backward pass so do the column sums of dgamma and
//     dbeta.  Each workgroup writes its sums once, to the workspace, and a
//     second kernel adds them in a fixed order: no atomics, the same bits on
//     every call.
//   * Rows of any width: the vectors are loaded from wherever the row starts
//     (global loads take any element alignment), and a row's last vector
//     element by element where it is not whole.
// Sums, statistics and weight gradients are fp32.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

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

// the vector of a row that starts at element c (c < cols); elements past the
// row's end are 0
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int c, int cols, float (&v)[Vec<T>::kN]) {
  constexpr int N = Vec<T>::kN;
  if (c + N <= cols) {
    const u32x4 w = *reinterpret_cast<const typename Vec<T>::raw*>(row + c);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (N == 8) v[i] = __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
      else v[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0f;
      if (c + i < cols) {
        if constexpr (N == 8) v[i] = bf16_to_f32(row[c + i]);
        else v[i] = row[c + i];
      }
    }
  }
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
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c + i < cols) {
        if constexpr (N == 8) row[c + i] = f32_to_bf16(v[i]);
        else row[c + i] = v[i];
      }
    }
  }
}

// N elements of an fp32 row vector of the weight's length; null: `fill`
template <int N>
__device__ __forceinline__ void load_weight(const float* w, int c, int cols, float fill, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = w != nullptr && c + i < cols ? w[c + i] : fill;
}

// sums of K values over the WPR waves of a row's group; every thread gets them
template <int WPR, int K>
__device__ __forceinline__ void group_sum(float (&s)[K], float* red) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += __shfl_xor(s[k], d);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;                   // a group is the whole workgroup
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

constexpr int threads_of(int wpr) { return wpr > 4 ? 64 * wpr : 256; }
constexpr int groups_of(int wpr) { return threads_of(wpr) / (64 * wpr); }     // rows at a time per workgroup

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
  int64_t rows;
  int cols;
  int layer;
  float eps;
};

template <typename T, int CH, int WPR>
__global__ __launch_bounds__(threads_of(WPR)) void norm_forward_kernel(NormArgs a) {
  constexpr int N = Vec<T>::kN, kT = 64 * WPR, kG = groups_of(WPR);
  __shared__ float red[WPR];
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
      group_sum<WPR, 1>(s, red);
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
    group_sum<WPR, 1>(q, red);
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

template <typename T, int CH, int WPR, bool BETA>
__global__ __launch_bounds__(threads_of(WPR)) void norm_backward_kernel(NormArgs a) {
  constexpr int N = Vec<T>::kN, kT = 64 * WPR, kG = groups_of(WPR);
  __shared__ float red[2 * WPR];
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
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kG + grp; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kG) {
    const size_t at = static_cast<size_t>(row) * cols;
    float h[CH][N], g[CH][N];
    const float mean = a.layer ? a.mean[row] : 0.0f, rstd = a.rstd[row];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * kT + t) * N;
      if (c < cols) {
        load_vec<T>(static_cast<const T*>(a.x) + at, c, cols, h[k]);
        load_vec<T>(static_cast<const T*>(a.dy) + at, c, cols, g[k]);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) h[k][i] = g[k][i] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // (past the row's end g is 0, so h adds nothing there)
        h[k][i] = (h[k][i] - mean) * rstd;
        dg[k][i] = fmaf(g[k][i], h[k][i], dg[k][i]);
        if constexpr (BETA) db[k][i] += g[k][i];
        g[k][i] *= gm[k][i];
        s[0] = fmaf(g[k][i], h[k][i], s[0]);
        s[1] += g[k][i];
      }
    group_sum<WPR, 2>(s, red);
    const float mh = s[0] * inv, m1 = a.layer ? s[1] * inv : 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (k * kT + t) * N;
      if (c < cols) {
        float r[N];
        if (a.residual != nullptr) {
          load_vec<T>(static_cast<const T*>(a.residual) + at, c, cols, r);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) r[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = fmaf(rstd, g[k][i] - m1 - h[k][i] * mh, r[i]);
        store_vec<T>(static_cast<T*>(a.y) + at, c, cols, r);
      }
    }
  }
  if (a.part == nullptr) return;
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
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (c + i < cols) part[static_cast<size_t>(b) * cols + c + i] = v[i];
      }
    }
}

// out[c] = sum over workgroups of part[w][b][c], in order: 16 slices of the
// workgroups, then the slices
constexpr int kFoldCols = 64, kFoldSlices = 16;

__global__ __launch_bounds__(kFoldCols* kFoldSlices) void norm_fold_kernel(const float* part, int groups, int nb,
                                                                           int cols, float* dgamma, float* dbeta) {
  __shared__ float red[kFoldSlices][kFoldCols];
  const int c = blockIdx.x * kFoldCols + threadIdx.x % kFoldCols, sl = threadIdx.x / kFoldCols;
  const int b = blockIdx.y;
  float* out = b ? dbeta : dgamma;
  float s = 0.0f;
  if (c < cols)
    for (int w = sl; w < groups; w += kFoldSlices) s += part[(static_cast<size_t>(w) * nb + b) * cols + c];
  red[sl][threadIdx.x % kFoldCols] = s;
  __syncthreads();
  if (sl == 0 && c < cols && out != nullptr) {
    for (int i = 1; i < kFoldSlices; ++i) s += red[i][threadIdx.x];
    out[c] = s;
  }
}

// Vectors per thread and waves per row.  One wave per row needs no barrier;
// more waves per row spread the few rows of a decode batch.
struct NormForm {
  int ch, wpr;
};

NormForm form_of(int64_t rows, int cols, int n, bool backward) {
  const int vecs = (cols + n - 1) / n;
  auto fits = [&](int ch, int wpr) { return vecs <= ch * wpr * 64; };
  const int most = backward ? 2 : 4;
  if (rows >= 1024) {
    for (int ch = 1; ch <= most; ch *= 2)
      if (fits(ch, 1)) return {ch, 1};
  } else if (fits(1, 1)) {
    return {1, 1};
  }
  for (int ch = 1; ch <= (rows >= 1024 ? most : 1); ch *= 2)
    if (fits(ch, 4)) return {ch, 4};
  for (int ch = 1; ch <= 4; ch *= 2)
    if (fits(ch, 16)) return {ch, 16};
  return {0, 0};
}

int grid_of(int64_t rows, NormForm f, bool backward) {
  const int64_t need = (rows + groups_of(f.wpr) - 1) / groups_of(f.wpr);
  const int64_t most = backward ? (f.wpr == 16 ? 256 : 512) : (f.wpr == 16 ? 512 : 2048);
  return static_cast<int>(need < most ? need : most);
}

template <typename T, int CH, int WPR>
void launch_fwd(const NormArgs& a, int grid, hipStream_t st) {
  norm_forward_kernel<T, CH, WPR><<<grid, threads_of(WPR), 0, st>>>(a);
}

template <typename T, int CH, int WPR>
void launch_bwd(const NormArgs& a, int grid, bool beta, hipStream_t st) {
  if (beta) norm_backward_kernel<T, CH, WPR, true><<<grid, threads_of(WPR), 0, st>>>(a);
  else norm_backward_kernel<T, CH, WPR, false><<<grid, threads_of(WPR), 0, st>>>(a);
}

template <typename T, typename F>
void with_form(NormForm f, F&& go) {
#define MOE_NORM_CASE(CH, WPR) \
  if (f.ch == CH && f.wpr == WPR) return go(std::integral_constant<int, CH>{}, std::integral_constant<int, WPR>{});
  MOE_NORM_CASE(1, 1) MOE_NORM_CASE(2, 1) MOE_NORM_CASE(4, 1)
  MOE_NORM_CASE(1, 4) MOE_NORM_CASE(2, 4) MOE_NORM_CASE(4, 4)
  MOE_NORM_CASE(1, 16) MOE_NORM_CASE(2, 16)
  if constexpr (sizeof(T) == 4) { MOE_NORM_CASE(4, 16) }
#undef MOE_NORM_CASE
}

}  // namespace

size_t norm_workspace_bytes(int64_t rows, int cols) {
  // the most workgroups of any form, two sums each
  size_t most = 0;
  for (int n = 4; n <= 8; n += 4) {
    const NormForm f = form_of(rows, cols, n, true);
    const size_t b = static_cast<size_t>(grid_of(rows, f, true)) * 2 * cols * sizeof(float);
    most = b > most ? b : most;
  }
  return (most + 255) & ~static_cast<size_t>(255);
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
  const NormForm f = form_of(rows, cols, bf16 ? 8 : 4, false);
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
  const bool any = dgamma != nullptr || dbeta != nullptr, beta = dbeta != nullptr;
  a.part = any ? static_cast<float*>(workspace) : nullptr;
  int grid = 0;
  if (rows > 0) {
    const NormForm f = form_of(rows, cols, bf16 ? 8 : 4, true);
    grid = grid_of(rows, f, true);
    if (bf16) with_form<bf16_t>(f, [&](auto ch, auto w) { launch_bwd<bf16_t, ch(), w()>(a, grid, beta, st); });
    else with_form<float>(f, [&](auto ch, auto w) { launch_bwd<float, ch(), w()>(a, grid, beta, st); });
  }
  if (any)
    norm_fold_kernel<<<dim3((cols + kFoldCols - 1) / kFoldCols, beta ? 2 : 1), kFoldCols * kFoldSlices, 0, st>>>(
        static_cast<const float*>(workspace), grid, beta ? 2 : 1, cols, dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace moe
