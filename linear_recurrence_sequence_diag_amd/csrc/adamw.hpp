// adamw.hpp -- host-side launcher of the AdamW update of many tensors (internal to liblrscan).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lrscan.h"

namespace lrscan {

struct AdamwArgs {
    double rate, beta1, beta2, eps, weight_decay;
    int64_t step;             // used where step_dev is NULL
    const int64_t* step_dev;  // device, or NULL
    const float* grad_scale;  // device, or NULL for 1
};

constexpr int kAdamwGroup = 256;  // elements that share the scale of an 8-bit state
constexpr int kAdamwThreads = 256, kAdamwPerBlock = 4096;  // of a workgroup; its elements, all of them loaded first
// Workgroups whose work-items stay in 32 bits, and what a tensor may hold.
constexpr int64_t kAdamwMaxBlocks = ((int64_t)1 << 32) / kAdamwThreads - 1;
constexpr int64_t kAdamwMaxElems = kAdamwMaxBlocks * kAdamwPerBlock;

hipError_t launch_adamw(const lrscan_adamw_tensor* tensors, int64_t count, int dtype, int state_bits, bool masters,
                        const AdamwArgs& a, hipStream_t st);

}  // namespace lrscan
