// Which tiles the head's loss takes, in how many pieces of the vocabulary and parts of a
// reduction, and where its workspace holds what: decided on the host from the sizes
// alone (no HIP in here).
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace moe {

constexpr int kOrderCols = 128;          // columns of the vocabulary whose targets are listed together
constexpr int kHeadStage = 64;           // a stage of a product's reduction

// Tiles: 256 x 256 with one workgroup a CU, 128 x 128 with two, and low ones that
// leave small batches bound by the weights.
enum Tile { kRows32, kRows64, kMid, kWide };

constexpr int up(int n, int to) { return (n + to - 1) / to * to; }

// What a backward pass holds: P for a piece of the vocabulary of about 2^27 entries
// (268 MB; whole tiles; at least 8192 columns, under which dx's fp32 sums, read and
// written once a piece, would cost a third of its product), x transposed, dx's sums.
struct Plan {
  int piece;                // columns of a piece, a multiple of 256
  int ldt;                  // rows, rounded up to 64
  Tile tile;                // of dx's product
  int parts;                // parts of its reduction
  bool sums;                // dx through fp32 sums
  size_t p, xt, dx, rest, order, order_at, bytes;
};

inline int rows_of(Tile t) { return t == kRows32 ? 32 : (t == kRows64 ? 64 : (t == kMid ? 128 : 256)); }
inline int cols_of(Tile t) { return t == kMid ? 128 : 256; }

inline int64_t tiles_of(Tile t, int64_t M, int64_t N) {
  return (M + rows_of(t) - 1) / rows_of(t) * ((N + cols_of(t) - 1) / cols_of(t));
}

// Time of n tiles over K in us: rounds of what the CUs hold at once (two of 128 x 128
// a CU; a last round that leaves one a CU runs its tiles faster), each a start and an
// end and K's stages.  Measured on 8192 rows by 32768 columns: 540, 898, 1672 us at K
// = 1024, 2048, 4096 in 256 x 256 tiles (16 rounds), 550, 990, 2016 in 128 x 128
// (32 rounds).  At 384 x 100352 over 4096 the narrow tiles' finer rounds win (340 us
// against 397), at 1024 rows they lose (820 against 715).
inline double cost(Tile t, int64_t n, int64_t K) {
  if (t == kWide) return static_cast<double>((n + 255) / 256) * (7.4 + 0.0236 * K);
  const int64_t left = n % 512;
  return (n / 512 + (left == 0 ? 0.0 : (left <= 256 ? 0.65 : 1.0))) * (1.5 + 0.0150 * K);
}

inline Tile pick_square(int64_t M, int64_t N, int64_t K) {
  return cost(kMid, tiles_of(kMid, M, N), K) < cost(kWide, tiles_of(kWide, M, N), K) ? kMid : kWide;
}

// The tile of `width` columns of the logits (and of P): low ones where the batch is
// that small (bound by the reads of the weights), else the cheaper of the two others.
inline Tile tile_of_logits(int64_t rows, int64_t width, int64_t cols) {
  if (rows <= 32) return kRows32;
  if (rows <= 64) return kRows64;
  return pick_square(rows, width, cols);
}

// dx's product: its tile, and the parts of its reduction that fill the CUs
struct Split {
  Tile tile;
  int parts;
};

inline Split pick_split(int64_t M, int64_t N, int64_t K) {
  Split best{kWide, 1};
  double least = -1.0;
  for (Tile t : {kRows32, kRows64, kMid, kWide}) {
    if ((t == kRows32 && M > 32) || (t == kRows64 && M > 64)) continue;
    const int64_t tiles = tiles_of(t, M, N), most = K / (16 * kHeadStage);    // at least 16 stages each
    int64_t parts = (t == kWide ? 256 : 512) / tiles;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    // with what the parts write and the last kernel reads, at 4.9 TB/s
    const double c = cost(t, tiles * parts, K / parts) + static_cast<double>(parts) * M * N * 8 / 4.9e6;
    if (least < 0 || c < least) {
      least = c;
      best = Split{t, static_cast<int>(parts)};
    }
  }
  return best;
}

inline Plan plan(int rows, int cols, int vocab) {
  Plan q{};
  q.ldt = up(rows, 64);
  int64_t piece = (int64_t{1} << 27) / q.ldt / 256 * 256;
  if (piece < 8192) piece = 8192;
  if (piece > up(vocab, 256)) piece = up(vocab, 256);
  q.piece = static_cast<int>(piece);
  const Split split = pick_split(rows, cols, q.piece);
  q.tile = split.tile;
  q.parts = split.parts;
  q.sums = q.parts > 1 || q.piece < vocab;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) / 256 * 256;
    return here;
  };
  q.p = take(static_cast<size_t>(rows) * q.piece * 2);
  q.xt = take(static_cast<size_t>(cols) * q.ldt * 2);
  q.dx = take(q.sums ? static_cast<size_t>(q.parts) * tiles_of(q.tile, rows, cols) * rows_of(q.tile) * cols_of(q.tile) * 4 : 0);
  q.rest = take(static_cast<size_t>(rows) * 4);
  q.order = take(static_cast<size_t>(rows) * 4);
  q.order_at = take((static_cast<size_t>(vocab) / kOrderCols + 2) * 4);
  q.bytes = at;
  return q;
}

// The pieces: columns v0 .. min(v0 + q.piece, vocab) - 1, one after the other
inline int piece_width(const Plan& q, int v0, int vocab) { return vocab - v0 < q.piece ? vocab - v0 : q.piece; }

// dW's tile for one
inline Tile tile_of_dw(const Plan& q, int width, int cols) { return pick_square(width, cols, q.ldt); }

// the parts of dx's reduction over one (a short last piece may have fewer stages than parts)
inline int parts_of_dx(const Plan& q, int width) {
  const int stages = up(width, kHeadStage) / kHeadStage;
  return q.parts < stages ? q.parts : stages;
}

// Bounds of what the forward pass and a plan take that do not shrink as rows grow (a
// plan's own sizes may: more rows can take shorter pieces and fewer parts).
inline size_t workspace_bound(int64_t rows, int cols, int vocab) {
  const size_t n = static_cast<size_t>(rows), V = static_cast<size_t>(up(vocab, 256));
  const size_t tiles = static_cast<size_t>(up(static_cast<int>(rows), 256)) * up(cols, 256);
  auto least = [](size_t a, size_t b) { return a < b ? a : b; };
  auto most = [](size_t a, size_t b) { return a > b ? a : b; };
  auto padded = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
  const size_t p = least(n * V, most(size_t{1} << 27, n * 8192)) * 2;
  // one part a tile, or as many as the CUs hold (at most 256 x 256 values each) with
  // 1024 columns each
  const size_t dx = most(tiles, least(size_t{256} << 16, tiles * (V / 1024))) * 4;
  const size_t backward = padded(p) + padded(static_cast<size_t>(cols) * up(static_cast<int>(rows), 64) * 2) + padded(dx) +
                          2 * padded(n * 4) + padded((static_cast<size_t>(vocab) / kOrderCols + 2) * 4);
  const size_t forward = n * ((vocab + 127) / 128 * size_t{8} + 4) + 512;    // (128: the narrowest tile's columns)
  return padded(most(forward, backward));
}

}  // namespace moe
