// Declarations of the output head's loss (head_loss.hip).
#pragma once

#include "moe_internal.h"

namespace moe {

size_t head_loss_workspace_bytes(int64_t rows, int cols, int vocab);
hipError_t launch_head_loss_forward(int rows, int cols, int vocab, const bf16_t* x, const bf16_t* w,
                                    const int32_t* target, float* loss, float* lse, void* workspace, hipStream_t st);
hipError_t launch_head_loss_backward(int rows, int cols, int vocab, const bf16_t* x, const bf16_t* w,
                                     const int32_t* target, const float* lse, const float* dloss, bf16_t* dx,
                                     bf16_t* dw, void* workspace, hipStream_t st);

}  // namespace moe
