// column_sum.hpp -- column sums of a [R, C] fp32 array of partial sums, in an
// order that R and C alone fix (results do not depend on scheduling).
// Internal to liblrscan; every translation unit that includes it gets its own
// copy (anonymous namespace).
//
// A workgroup owns 64 columns and a range of rows: wavefront w adds rows w,
// w + 16, ... of the range, four at a time, and the 16 sums are added in order
// through LDS.  Where the rows are many and the columns few, the ranges'
// sums go to `scratch` and are added by a second launch.  `Write::put(c, sum)`
// receives the result of column c.  A launch and one round of loads bound it:
// 4 to 5 us for 64 rows of 2560 columns and for 72 of 12800.
#pragma once

#include "device.hpp"

namespace lrscan {

namespace {

constexpr int kSumWaves = 16;
constexpr int64_t kSumRows = 512;  // rows of a range
constexpr int kSumRanges = 64;     // at most

template <class Write>
__global__ __launch_bounds__(kSumWaves* kWave) void column_sum_kernel(const float* part, int64_t R,
                                                                      int64_t C, int64_t per, Write out) {
    __shared__ float s_sum[kSumWaves][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWave + lane;
    const int64_t r0 = (int64_t)blockIdx.y * per;
    const int64_t r1 = r0 + per < R ? r0 + per : R;
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < C) {
        int64_t r = r0 + wave;
        for (; r + 3 * kSumWaves < r1; r += 4 * kSumWaves) {
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] += part[(size_t)(r + q * kSumWaves) * C + c];
        }
        for (; r < r1; r += kSumWaves) a[0] += part[(size_t)r * C + c];
    }
    s_sum[wave][lane] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (wave == 0 && c < C) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWaves; ++w) t += s_sum[w][lane];
        out.put((int64_t)blockIdx.y, c, t);
    }
}

// Range sums into rows of a [ranges, C] array.
struct WriteRows {
    float* p;
    int64_t C;
    __device__ __forceinline__ void put(int64_t row, int64_t c, float x) const { p[(size_t)row * C + c] = x; }
};

int64_t column_sum_ranges(int64_t R) {
    const int64_t n = (R + kSumRows - 1) / kSumRows;
    return n < kSumRanges ? n : kSumRanges;
}

// Whether a launch's work-items along the columns stay in 32 bits.
bool column_sum_fits(int64_t C) {
    return (C + kWave - 1) / kWave < ((int64_t)1 << 32) / (kSumWaves * kWave);
}

// Bytes of `scratch` (0 if one launch does).
size_t column_sum_scratch(int64_t R, int64_t C) {
    const int64_t n = column_sum_ranges(R);
    return n > 1 ? (size_t)n * (size_t)C * 4 : 0;
}

template <class Write>
hipError_t launch_column_sum(const float* part, int64_t R, int64_t C, float* scratch, Write out,
                             hipStream_t st) {
    const int64_t n = column_sum_ranges(R), per = (R + n - 1) / n;
    const dim3 block(kSumWaves * kWave);
    const unsigned cols = (unsigned)((C + kWave - 1) / kWave);
    if (n > 1) {
        hipLaunchKernelGGL((column_sum_kernel<WriteRows>), dim3(cols, (unsigned)n), block, 0, st, part, R,
                           C, per, WriteRows{scratch, C});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((column_sum_kernel<Write>), dim3(cols, 1), block, 0, st, scratch, n, C, n, out);
    } else {
        hipLaunchKernelGGL((column_sum_kernel<Write>), dim3(cols, 1), block, 0, st, part, R, C, R, out);
    }
    return hipGetLastError();
}

}  // namespace

}  // namespace lrscan
