// delta_blocks.hpp -- gated delta rule: blocks of tokens, parts of a row, and the
// places of what passes between blocks.  Plain integer code, apart from the
// kernels so that it can be checked on the host.
#pragma once

#include <stdint.h>

namespace lrscan {
namespace delta {

constexpr int kC = 64;  // tokens of a block
constexpr int kCut = (int)0x80000000;

// ---- the blocks of a batch row ----
// Every block of up to kC tokens lies within one segment, so no product reaches
// from one segment into another.  Without resets they start at multiples of kC.
struct Blocks {
    const int* starts;  // [B][T + 1], kCut set where a segment starts, the last one T; NULL without resets
    const int* counts;  // [B]
    int T;
    __host__ __device__ __forceinline__ int count(int64_t b) const { return starts ? counts[b] : (T + kC - 1) / kC; }
    // block c, and whether a reset starts it
    __host__ __device__ __forceinline__ void at(int64_t b, int c, int& start, int& len, bool& cut) const {
        if (starts) {
            const int* p = starts + b * ((int64_t)T + 1) + c;
            cut = p[0] < 0;
            start = p[0] & ~kCut;
            len = (p[1] & ~kCut) - start;
        } else {
            start = c * kC;
            len = T - start < kC ? T - start : kC;
            cut = false;
        }
    }
    // whether a reset starts the block behind c, of n
    __host__ __device__ __forceinline__ bool cut_behind(int64_t b, int c, int n) const {
        bool cut = false;
        int start, len;
        if (c + 1 < n) at(b, c + 1, start, len, cut);
        return cut;
    }
};

// The first block of a part, of n blocks in `parts`; its end is the next one's.
__host__ __device__ __forceinline__ int part_start(int n, int part, int parts) { return (int)((int64_t)n * part / parts); }

// States at the blocks' starts: a block that a segment does not start begins 64
// tokens behind another of its segment, so start / 64 is its own slot; one more
// for the sequence's end.  Of a block that a segment starts it may be another's,
// so what enters such a block is written nowhere.
__host__ __device__ __forceinline__ int64_t state_slots(int64_t T) { return T / kC + 2; }
// The slot of what enters a block from `start` on, and of what leaves one in front of `behind`.
__host__ __device__ __forceinline__ int64_t entering_slot(int start) { return start / kC; }
__host__ __device__ __forceinline__ int64_t leaving_slot(int64_t T, int behind) {
    return behind < T ? behind / kC : state_slots(T) - 1;
}

}  // namespace delta
}  // namespace lrscan
