// delta.hpp -- host-side launchers of the gated delta rule (internal to liblrscan).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lrscan {

// Rows of one [B, T, heads, width] operand: base pointer and the byte distances
// between batch rows, steps and heads (the last dimension is contiguous).
struct HeadRows {
    char* p;
    int64_t sb, st, sh;
    __device__ __forceinline__ char* row(int64_t b, int64_t t, int64_t h) const {
        return p + b * sb + t * st + h * sh;
    }
};

struct DeltaShape {
    int64_t B, T;
    int H, HK, K, V;  // value heads, query/key heads, rows and columns of a head's state
    int dtype;        // DT_F32 / DT_BF16
};

struct DeltaIn {
    HeadRows q, k, v;
    HeadRows g, beta;  // [B, T, H] fp32
    float scale;
    const float* h0;   // [B, H, K, V] or NULL
    const uint8_t* reset;
};

struct DeltaFwd {
    void* out;    // [B, T, H, V] or NULL
    float* last;  // [B, H, K, V] or NULL
};

struct DeltaBwd {
    const void* grad_out;    // [B, T, H, V], contiguous as every gradient
    const float* grad_last;  // or NULL
    void *grad_q, *grad_k, *grad_v;
    float *grad_g, *grad_beta;
    float* grad_h0;  // or NULL
};

constexpr int kDeltaMaxK = 256;

// Whether the shape's launches and offsets fit what the kernels count with.
enum DeltaPass { kDeltaForward, kDeltaBackward, kDeltaStep };
bool delta_fits(const DeltaShape& s, DeltaPass pass, bool reset);
// Scratch of a call (256-byte aligned; rewritten before it is read), or (in NULL)
// of the call with the largest of any operands of these sizes; grad_out: of a backward.
size_t delta_ws_bytes(const DeltaShape& s, const DeltaIn* in, const void* grad_out, bool backward);
hipError_t launch_delta_fwd(const DeltaShape& s, const DeltaIn& in, const DeltaFwd& p, void* ws, hipStream_t st);
hipError_t launch_delta_bwd(const DeltaShape& s, const DeltaIn& in, const DeltaBwd& p, void* ws, hipStream_t st);
// One token: in.h0 is the state that enters, in.reset [B].  `last` may be in.h0.
hipError_t launch_delta_step(const DeltaShape& s, const DeltaIn& in, const DeltaFwd& p, hipStream_t st);

}  // namespace lrscan
