// delta_ws.hpp -- the gated delta rule's scratch and the passes over it
// (internal to the delta_*.hip files).
#pragma once

#include "delta_tile.hpp"

namespace lrscan {
namespace delta {

// Elements of a row of n that is whole vectors of 16 bytes.
inline int row_width(int n, int dtype) {
    const int per = dtype == DT_F32 ? 4 : 8;
    return (n + per - 1) / per * per;
}
// Columns of the scratch rows that the backward keeps.
__host__ __device__ __forceinline__ int kept_width(int V) { return (V + 7) / 8 * 8; }

constexpr int kComputeUnits = 256;

// Parts of a sequence that are walked at the same time, where its heads leave most
// compute units idle.  Forming the parts' maps, of K + V columns, takes as long as
// the walk itself or longer, so it pays from three parts on whose maps find room at
// once, of three blocks or more each; joining them takes a step for each part, so
// there are no more than twice the root of the blocks.  us of a forward and of a
// reverse call without parts and with them, B = 1, K = V = 128, bf16:
//   8 heads, T = 800      70, 160     57, 142
//   8 heads, T = 2048    150, 314     80, 188
//   8 heads, T = 32768  2216, 5232   409, 1325
//  32 heads, T = 1024     87, 221     71, 207
//  43 heads, T = 2048    169, 548    177, 520 (in five parts, whose maps find no room at once)
inline int sequence_parts(const DeltaShape& d) {
    const int64_t units = d.B * d.H * ((d.K + d.V + 127) / 128), blocks = (d.T + kC - 1) / kC;
    int64_t parts = kComputeUnits / units < blocks / 3 ? kComputeUnits / units : blocks / 3;
    while (parts * parts > 4 * blocks) --parts;
    return parts < 3 ? 1 : (int)parts;
}

// Operands whose rows are not whole aligned vectors, or lie too far apart for
// 32-bit offsets within a block, are copied into rows that are.
struct Copies {
    bool q, k, v, go;
};
inline bool rows_whole(const HeadRows& r, int width, int bytes) {
    return (reinterpret_cast<uintptr_t>(r.p) | (uintptr_t)r.sb | (uintptr_t)r.st | (uintptr_t)r.sh |
            (uintptr_t)(width * bytes)) % 16 == 0 &&
           r.st >= width * bytes && r.st <= (1 << 24);
}

// Byte offsets into a call's workspace.
struct Layout {
    size_t starts, counts, gates, gl, inv, att, att_t, inv_t, x, r, s, ds, sums, between, behind, map, map_t, q, k, v, go, total;
    Layout(const DeltaShape& d, bool backward, bool reset, const Copies& copy) {
        const size_t tokens = (size_t)d.B * d.H * d.T, bytes = d.dtype == DT_F32 ? 4 : 2;
        size_t at = 0;
        auto take = [&](size_t& o, size_t n, bool wanted) {
            o = at;
            if (wanted) at += (n + 255) / 256 * 256;
        };
        take(starts, (size_t)d.B * (d.T + 1) * 4, reset);
        take(counts, (size_t)d.B * 4, reset);
        take(gates, tokens * 16, true);
        take(gl, tokens * 4, backward);
        take(inv, tokens * kC * 6, true);
        take(att, tokens * kC * 6, !backward);
        take(att_t, tokens * kC * 6, backward);
        take(inv_t, tokens * kC * 6, backward);
        take(x, tokens * kept_width(d.V) * 4, backward);
        take(r, tokens * kept_width(d.V) * 4, backward);
        const size_t state = (size_t)d.B * d.H * state_slots(d.T) * d.K * kept_width(d.V) * 4;
        take(s, state, backward);
        take(ds, state, backward);
        take(sums, (size_t)d.B * d.HK * ((d.T + kC - 1) / kC) * kGradThreads * 8 * 16, backward && d.H > d.HK);
        const int64_t parts = sequence_parts(d);
        const size_t heads = (size_t)d.B * d.H * parts;
        take(between, heads * d.K * kept_width(d.V) * 4, parts > 1);
        take(behind, heads * d.K * kept_width(d.V) * 4, parts > 1 && backward);
        take(map, heads * d.K * kept_width(d.K) * 4, parts > 1);
        take(map_t, heads * d.K * kept_width(d.K) * 4, parts > 1 && backward);
        const size_t kr = (size_t)d.B * d.T * d.HK * row_width(d.K, d.dtype) * bytes, vr = tokens * row_width(d.V, d.dtype) * bytes;
        take(q, kr, copy.q);
        take(k, kr, copy.k);
        take(v, vr, copy.v);
        take(go, vr, backward && copy.go);
        total = at;
    }
};

// What the backward keeps between its passes, in fp32, in rows of kept_width(V).
struct Kept {
    float *x, *r;   // [B, H, T]: x of the forward, and the gradient of beta (x's right side)
    float *s, *ds;  // [B, H, slots, K]: states that enter blocks, gradients that leave them
    f32x4* sums;    // a workgroup's kGradThreads x 8: of q's and k's gradients over the heads that share a q and k so far
};

// Between the parts of a sequence, in fp32, [B, H, parts]: the state that enters a
// part and the gradient of the one that leaves it (rows of kept_width(V)); the
// parts' maps, and transposed (rows of kept_width(K)).
struct Parts {
    int n;
    float *enter, *leave, *map, *map_t;
};

// Copies of rows [B, T, heads, n] into contiguous ones of `width`, zeros behind.
struct RowCopies {
    struct One {
        HeadRows from;
        void* to;
        int64_t heads, rows;
        int n, width;
    } of[4];
    int count;
};
hipError_t run_copies(const RowCopies& copies, int64_t T, int dtype, hipStream_t st);
hipError_t run_blocks(const DeltaShape& s, const uint8_t* reset, int* starts, int* counts, hipStream_t st);
hipError_t run_prep(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, bool backward,
                    hipStream_t st);
// The walk over the blocks: outputs and the last state, or (keep) x and the entering states.
hipError_t run_walk(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                    const DeltaFwd& out, const Kept* keep, const Parts& parts, hipStream_t st);
// The walk back: r, grad_v, the gradients that leave blocks, and grad_h0.
hipError_t run_walk_back(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                         const DeltaBwd& p, const HeadRows& go, const Kept& keep, const Parts& parts, hipStream_t st);
// The other gradients, every block by itself.
hipError_t run_grads(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                     const DeltaBwd& p, const HeadRows& go, const Kept& keep, hipStream_t st);

}  // namespace delta
}  // namespace lrscan
