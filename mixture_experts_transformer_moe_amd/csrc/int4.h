// Declarations of the experts' products with 4-bit weights (int4.hip).
#pragma once

#include "moe_internal.h"

namespace moe {

hipError_t launch_quantize_int4(const bf16_t* src, uint8_t* dst, bf16_t* scales, int64_t count, int rows, int cols,
                                int group, hipStream_t st);
hipError_t launch_pack_int4(const uint8_t* codes, uint8_t* dst, int64_t count, int rows, int cols, hipStream_t st);
hipError_t launch_gate_up_int4(const moe_shape& s, int group, const bf16_t* x_perm, const int32_t* sorted_token,
                               const bf16_t* x, const int32_t* offsets, const uint8_t* wgu, const bf16_t* sgu,
                               const uint8_t* wsgu, const bf16_t* ssgu, bf16_t* h, hipStream_t st);
hipError_t launch_down_int4(const moe_shape& s, int group, const bf16_t* h, const int32_t* offsets,
                            const uint8_t* wd, const bf16_t* sd, const uint8_t* wsd, const bf16_t* ssd,
                            bf16_t* y_perm, bf16_t* y_shared, hipStream_t st);

}  // namespace moe
