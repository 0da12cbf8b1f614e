// logits.hpp -- host-side launcher of the adjustment of logits (internal to liblrscan).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lrscan {

struct LogitsArgs {
    const void* in;
    void* out;  // may be `in`
    int64_t B, V, in_stride, out_stride;
    int dtype, id_bytes;
    const void* tokens;  // [B] rows of L, `token_stride` apart, or NULL
    int64_t L, token_stride;
    const void *lengths, *prompts;                      // [B] or NULL
    const float *repetition, *presence, *frequency;     // [B] or NULL
    const void* bias_ids;                               // [B, K] or NULL
    const float* bias;
    int64_t K;
    const uint32_t* allowed;  // [B, ceil(V / 32)] or NULL
};

bool logits_fits(const LogitsArgs& a);
hipError_t launch_logits(const LogitsArgs& a, hipStream_t st);

}  // namespace lrscan
