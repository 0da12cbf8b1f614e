// gated.hpp -- host-side launchers of the gated scan (internal to liblrscan).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lrscan {

// Rows of one [B, T, D] operand: base pointer and the byte distances between
// its batch rows and between its steps (the last dimension is contiguous).
struct Rows {
    char* p;
    size_t sb, st;
    __device__ __forceinline__ char* row(int64_t b, int64_t t) const {
        return p + (size_t)b * sb + (size_t)t * st;
    }
};

struct GatedShape {
    int64_t B, T, D;
    int dtype;  // DT_F32 / DT_BF16
};

struct GatedFwd {
    Rows x, gr, gi;
    const float* decay;
    float scale;
    void* out;    // contiguous, or NULL (state only)
    float* last;  // may be h0 itself where T = 1
    const float* h0;
    const uint8_t* reset;
};

struct GatedBwd {
    Rows x, gr, gi;
    const float* decay;
    float scale;
    const void *out, *g;  // contiguous
    const float *grad_last, *h0;
    const uint8_t* reset;
    Rows gx, ggr, ggi;
    float* grad_h0;
};

// Whether every row of an operand starts 16-byte aligned (its rows' length
// aside), and of every operand of a call.
bool operand_aligned(int64_t B, int64_t T, const Rows& r);
bool gated_fwd_aligned(const GatedShape& s, const GatedFwd& p);
bool gated_bwd_aligned(const GatedShape& s, const GatedBwd& p);

// The per-lane walk.  A thread walks gated_walk_rows batch rows; the backward's
// `part` (or NULL) receives a row of D partial sums of P from each such group.
int64_t gated_walk_rows(const GatedShape& s);
bool gated_walk_fits(const GatedShape& s);
hipError_t launch_gated_walk_fwd(const GatedShape& s, const GatedFwd& p, hipStream_t st);
hipError_t launch_gated_walk_bwd(const GatedShape& s, const GatedBwd& p, float* part, hipStream_t st);

// The tiled single-launch form (scratch conventions of the fused form).  It
// takes a shape whose tiles' byte offsets stay in 32 bits, `row_strides` the
// bytes between the steps of its strided operands.  The backward's `part` (or
// NULL) receives gated_fused_part_rows rows of D partial sums of P.
bool gated_fused_fits(const GatedShape& s, int dir, const size_t* row_strides, int n);
size_t gated_fused_bytes(const GatedShape& s);
int64_t gated_fused_part_rows(const GatedShape& s);
hipError_t launch_gated_fused_fwd(const GatedShape& s, const GatedFwd& p, void* ws, size_t ws_bytes,
                                  bool init, int polls, hipStream_t st);
hipError_t launch_gated_fused_bwd(const GatedShape& s, const GatedBwd& p, float* part, void* ws,
                                  size_t ws_bytes, bool init, int polls, hipStream_t st);

// grad_decay from `rows` rows of D partial sums; `scratch` holds
// gated_decay_scratch bytes.
bool gated_decay_fits(int64_t D);
size_t gated_decay_scratch(int64_t rows, int64_t D);
hipError_t launch_gated_decay(const float* part, int64_t rows, int64_t D, float* scratch,
                              const float* decay, float* grad_decay, hipStream_t st);

}  // namespace lrscan
