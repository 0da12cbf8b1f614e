// conv.hpp -- host-side launchers of the short causal convolution (internal to
// liblrscan).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gated.hpp"

namespace lrscan {

constexpr int kMinTaps = 2, kMaxTaps = 4;

struct ConvShape {
    int64_t B, T, D;
    int K;      // taps
    int dtype;  // DT_F32 / DT_BF16
    int silu;   // 1: y = z sigmoid(z), 0: y = z
};

struct ConvFwd {
    Rows x;
    const float *w, *bias;  // [K, D]; [D] or NULL
    const void* state;      // [B, K - 1, D] inputs before the first, or NULL
    const uint8_t* reset;
    void* out;              // contiguous
    void* last;             // [B, K - 1, D], or NULL; may be `state` where T = 1
};

struct ConvBwd {
    Rows x;
    const float *w, *bias;
    const void* state;
    const uint8_t* reset;
    const void *g, *grad_last;  // contiguous; [B, K - 1, D] or NULL
    Rows gx;
    void* grad_state;  // [B, K - 1, D] or NULL
};

// Whether a backward can have parameter gradients, and the bytes of their
// partial sums and of the reduction's scratch.
bool conv_sums_fit(const ConvShape& s);
size_t conv_part_bytes(const ConvShape& s);
size_t conv_sum_scratch(const ConvShape& s);
bool conv_fits(const ConvShape& s);
hipError_t launch_conv_fwd(const ConvShape& s, const ConvFwd& p, hipStream_t st);
// `part` is NULL when neither grad_w nor grad_bias is wanted.
hipError_t launch_conv_bwd(const ConvShape& s, const ConvBwd& p, float* part, float* scratch,
                           float* grad_w, float* grad_bias, hipStream_t st);

}  // namespace lrscan
