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
// Numbers.  A code is stored as q + 8; 128 + (q + 8) is a bf16 whose low mantissa
// bits are the code, so eight codes become an MFMA operand with four AND-ORs and
// three shifts, no conversion.  The offset leaves again through the accumulator:
// a group's MFMA chain starts from -136 sum_{c in g} a[p, c], itself an MFMA
// chain with a constant operand, shared by all weight rows of the wave.  The
// products are exact, the sums fp32; the offset makes their rounding about 30
// times that of a plain fp32 sum (2e-6 of a group's result, against 2^-8 of the
// bf16 output).  A group's sum is then multiplied by its scale in fp32.
//
// Layout.  Blocks of 16 rows x 128 columns, 1 KB, row-block major: lane l's 16
// bytes are its codes of four 16x16x32 MFMA steps, row l mod 16, columns
// 32 i + 8 (l / 16) .. + 7 of dword i, element e in nibble e / 2 + 4 (e mod 2)
// (so that one mask takes out elements 2j and 2j + 1 as a bf16 pair).
#include "int4.h"

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

// eight codes -> the bf16 operand 128 + code (element e from nibble e / 2 + 4 (e mod 2))
__device__ __forceinline__ bf16x8 widen(uint32_t w) {
  constexpr uint32_t kMask = 0x000f000fu, kBase = 0x43004300u;
  const u32x4 v = {(w & kMask) | kBase, ((w >> 4) & kMask) | kBase, ((w >> 8) & kMask) | kBase,
                   ((w >> 12) & kMask) | kBase};
  return __builtin_bit_cast(bf16x8, v);
}

// One workgroup: a column tile of one expert, its rows 16 TB at a time.  Four
// waves of 64 weight rows each (gate_up: 32 gate rows and the up rows of the same
// columns): ks of them share the reduction, 4 / ks stand side by side.
template <int MODE, int TB, int G>
__global__ __launch_bounds__(256, TB <= 2 ? 3 : 2) void int4_rows_kernel(Int4Args a) {
  constexpr int NB = 4;                                   // 16-row weight blocks of a wave
  constexpr int kCols = MODE == kInt4GateUp ? 32 : 64;    // output columns of a wave
  constexpr int GC = kColBlock / G;                       // groups of a packed block
  __shared__ __attribute__((aligned(16))) float part[4 * NB * TB * 256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // ---- whose tile: the shared expert's first, then those of the experts with rows
  int bid = blockIdx.x;
  const bool shared = bid < a.tiles_s;
  int e = 0, lo = 0, M = a.T, tile = bid;
  if (!shared) {
    bid -= a.tiles_s;
    int slot = bid / a.tiles_r;
    tile = bid % a.tiles_r;
    e = -1;
    for (int c = 0; c < a.E; c += 64) {
      const int i = c + lane;
      // clamped so that no offsets table can move a row outside [0, S)
      const int from = min(max(a.offsets[min(i, a.E)], 0), a.S);
      const int to = min(max(a.offsets[min(i + 1, a.E)], from), a.S);
      const bool has = i < a.E && to > from;
      const uint64_t m = __ballot(has);
      const int n = __popcll(m);
      if (slot < n) {
        const int rank = __popcll(m & ((uint64_t{1} << lane) - 1));
        const int src = __ffsll(static_cast<unsigned long long>(__ballot(has && rank == slot))) - 1;
        e = __builtin_amdgcn_readfirstlane(c + src);
        lo = __builtin_amdgcn_readlane(from, src);
        M = __builtin_amdgcn_readlane(to, src) - lo;
        break;
      }
      slot -= n;
    }
    if (e < 0) return;
  }
  const int K = shared ? a.Ks : a.K;
  const int N = shared ? a.Ns : a.N;
  const int ks = shared ? a.ks_s : a.ks_r;
  const int rs = 4 / ks;
  const int Nw = MODE == kInt4GateUp ? 2 * N : N;
  const int ncb = K / kColBlock;
  const int kpart = wave % ks, side = wave / ks;
  const int c0 = ncb * kpart / ks, c1 = ncb * (kpart + 1) / ks;
  const int n0 = (tile * rs + side) * kCols;

  // ---- weights and scales of the wave's four blocks
  const uint8_t* wmat = shared ? a.w_shared : a.w_routed + static_cast<size_t>(e) * Nw * (K / 2);
  const bf16_t* smat = shared ? a.s_shared : a.s_routed + static_cast<size_t>(e) * Nw * (K / G);
  auto block_row = [&](int b) {
    return MODE == kInt4GateUp ? (b < 2 ? n0 + 16 * b : N + n0 + 16 * (b - 2)) : n0 + 16 * b;
  };
  const uint8_t* wb[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    wb[b] = wmat + static_cast<size_t>(block_row(b) / kRowBlock) * ncb * kBlockBytes + lane * 16;
  // lane l loads the scale of row l of the wave's 64
  const int sb = lane >> 4;
  const int srow = (MODE == kInt4GateUp ? (sb < 2 ? n0 + 16 * sb : N + n0 + 16 * (sb - 2)) : n0 + 16 * sb) + (lane & 15);
  const bf16_t* sp = smat + static_cast<size_t>(srow) * (K / G);

  struct Buf {
    u32x4 w[NB];
    u32x4 x[TB][4];
    uint16_t s[GC];
  };

  for (int m0 = 0; m0 < M; m0 += 16 * TB) {
    const bf16_t* xr[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const int m = min(m0 + 16 * t + (lane & 15), M - 1);
      const bf16_t* base = a.a_shared;
      int row = m;
      if (!shared) {
        base = a.a_routed;
        row = lo + m;
        if (a.gather) row = min(max(a.gather[row], 0), a.T - 1);
      }
      xr[t] = base + static_cast<size_t>(row) * K + 8 * (lane >> 4);
    }
    f32x4 acc[TB][NB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto load = [&](Buf& f, int cb) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        f.w[b] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wb[b] + static_cast<size_t>(cb) * kBlockBytes));
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f.x[t][i] = *reinterpret_cast<const u32x4*>(xr[t] + cb * kColBlock + 32 * i);
#pragma unroll
      for (int g = 0; g < GC; ++g) f.s[g] = sp[cb * GC + g];
    };
    auto compute = [&](const Buf& f) __attribute__((always_inline)) {
      constexpr int SG = 4 / GC;                         // MFMA steps of a group
      const u32x4 offset = {0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u};   // -136
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        // the scales of rows l mod 16 of each block, from the lanes that loaded them
        const uint32_t own = static_cast<uint32_t>(f.s[g]) << 16;
        const auto p = __builtin_amdgcn_permlane32_swap(own, own, false, false);       // rows 0 1 0 1, 2 3 2 3
        const auto p01 = __builtin_amdgcn_permlane16_swap(p[0], p[0], false, false);
        const auto p23 = __builtin_amdgcn_permlane16_swap(p[1], p[1], false, false);
        const float sc[NB] = {__uint_as_float(p01[0]), __uint_as_float(p01[1]), __uint_as_float(p23[0]),
                              __uint_as_float(p23[1])};
        f32x4 base[TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          base[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < SG; ++i)
            base[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.x[t][g * SG + i]),
                                                               __builtin_bit_cast(bf16x8, offset), base[t], 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          bf16x8 w[SG];
#pragma unroll
          for (int i = 0; i < SG; ++i) w[i] = widen(f.w[b][g * SG + i]);
#pragma unroll
          for (int t = 0; t < TB; ++t) {
            f32x4 y = base[t];
#pragma unroll
            for (int i = 0; i < SG; ++i)
              y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.x[t][g * SG + i]), w[i], y, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][b][r] = fmaf(sc[b], y[r], acc[t][b][r]);
          }
        }
      }
    };
    // two buffers; the loads are unconditional (the last repeats a block), so that
    // the waits before each block leave the next one's loads in flight
    if (c0 < c1) {
      Buf f0, f1;
      load(f0, c0);
      for (int cb = c0;;) {
        load(f1, min(cb + 1, c1 - 1));
        compute(f0);
        if (++cb >= c1) break;
        load(f0, min(cb + 1, c1 - 1));
        compute(f1);
        if (++cb >= c1) break;
      }
    }

    // ---- the waves' parts meet in LDS: [wave][tb][block][token][row]
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          part[((wave * TB + t) * NB + b) * 256 + (4 * (lane >> 4) + r) * 16 + (lane & 15)] = acc[t][b][r];
    __syncthreads();
    const int pairs = kCols / 2;                          // column pairs of a side
    for (int i = tid; i < rs * 16 * TB * pairs; i += 256) {
      const int c = 2 * (i % pairs), rest = i / pairs;
      const int m = rest % (16 * TB), sd = rest / (16 * TB);
      if (m0 + m >= M) continue;
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
    __syncthreads();
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

template <int MODE, int G>
hipError_t launch_rows(Int4Args a, int slots, int tb, hipStream_t st) {
  constexpr int kCols = MODE == kInt4GateUp ? 32 : 64;
  const unsigned grid = static_cast<unsigned>(a.tiles_s) + static_cast<unsigned>(slots) * a.tiles_r;
  (void)kCols;
  if (grid == 0) return hipSuccess;
  if (tb == 1) int4_rows_kernel<MODE, 1, G><<<grid, 256, 0, st>>>(a);
  else if (tb == 2) int4_rows_kernel<MODE, 2, G><<<grid, 256, 0, st>>>(a);
  else int4_rows_kernel<MODE, 4, G><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_int4(Int4Args a, const moe_shape& s, int group, hipStream_t st) {
  constexpr int kCols = MODE == kInt4GateUp ? 32 : 64;
  const int slots = a.S < a.E ? a.S : a.E;
  // waves that share a reduction: one, unless too few workgroups would be left
  auto split = [&](int K, int N, int groups) {
    int ks = 1;
    while (ks < 4 && K / kColBlock >= 4 * ks && static_cast<int64_t>(groups) * (N / (kCols * (4 / ks))) < 2048) ks *= 2;
    return ks;
  };
  a.ks_r = split(a.K, a.N, slots);
  a.tiles_r = a.N / (kCols * (4 / a.ks_r));
  a.ks_s = a.Ns > 0 ? split(a.Ks, a.Ns, 1) : 1;
  a.tiles_s = a.Ns > 0 ? a.Ns / (kCols * (4 / a.ks_s)) : 0;
  const int mean = a.S / a.E;
  const int tb = mean >= 48 ? 4 : (mean >= 8 || s.T > 16 ? 2 : 1);
  switch (group) {
    case 32: return launch_rows<MODE, 32>(a, slots, tb, st);
    case 64: return launch_rows<MODE, 64>(a, slots, tb, st);
    default: return launch_rows<MODE, 128>(a, slots, tb, st);
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
  return launch_int4<kInt4GateUp>(a, s, group, st);
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
  return launch_int4<kInt4Down>(a, s, group, st);
}

}  // namespace moe
