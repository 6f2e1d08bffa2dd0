// Which kernel the 4-bit products take: decided on the host from the sizes alone (no HIP
// in here).
#pragma once

#include <cstdint>

namespace moe {

enum class Int4Kernel { kRows16, kRows32, kTiles };

// By the mean rows an expert.  The tile kernel spreads a weight's conversion over
// 128 rows but streams weights more slowly; scales of 32 columns cost it more.
// Measured at D = 4096, F = 1024 (us: 16-row, 32-row and tile kernel), groups of 128:
// gate/up 230, 245, 301 at 12 rows, 259, 252, 316 at 14, 405, 315, 323 at 24, 454, 356,
// 328 at 28; down (K = 1024) 138, 148, 164 at 12, 150, 157, 165 at 14, 169, 166, 168 at
// 16, 186, 171, 167 at 18; groups of 32: gate/up 504, 405, 424 at 28, 560, 470, 441 at
// 32, down 224, 201, 203 at 20, 248, 217, 208 at 24.  The shared expert's T rows go
// with the routed ones.
inline Int4Kernel int4_kernel(bool gate_up, int group, int routed_rows, int experts) {
  const int mean = routed_rows / experts;
  const int tiles_from = gate_up ? (group == 32 ? 30 : 26) : (group == 32 ? 22 : 17);
  if (mean >= tiles_from) return Int4Kernel::kTiles;
  return mean >= 14 ? Int4Kernel::kRows32 : Int4Kernel::kRows16;
}

// Waves of a workgroup of the rows kernels that share a reduction.  More of them make more
// workgroups of the same rows, which evens out their last round; each costs a start
// (offsets, row ids, first loads: 4 to 6 us, beside the others').  So up to 4096
// workgroups as long as a wave keeps 8 blocks, and up to 1024 at any length (D = 4096,
// F = 1024, even popularity: 32 tokens' gate/up 118 us, 130 whole, 125 in fours; 1
// token's 14.5, 30 whole; 32 tokens' down, K = 1024, 66, 66 and 86).
// blocks: 128-column blocks of the reduction; columns: output columns of a wave
inline int int4_split(int blocks, int outputs, int columns, int64_t chunks) {
  int ks = 1;
  for (; ks < 4; ks *= 2) {
    const int64_t groups = chunks * (outputs / (columns * (4 / ks)));
    const int left = blocks / (2 * ks);                     // of a wave after one more split
    if (!(left >= 8 && groups < 4096) && !(left >= 2 && groups < 1024)) break;
  }
  return ks;
}

}  // namespace moe
