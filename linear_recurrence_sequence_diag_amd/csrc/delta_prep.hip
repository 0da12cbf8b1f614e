// delta_prep.hip -- gated delta rule: the blocks of a batch row, and what each
// block's walk needs that does not depend on the state.
//
// Within a block that starts from the state S, with G_i the running sum of
// log_decay, D_ij = exp(G_i - G_j) and u_j = beta_j x_j what token j adds,
//   x_i = v_i - exp(G_i) S^T k_i - sum_{j < i} D_ij (k_i.k_j) beta_j x_j,
// so X = (I + N)^-1 (V - diag(exp G) K S), N_ij = D_ij (k_i.k_j) beta_j below
// the diagonal.  The inverse is formed by substitution in the four 16x16 blocks
// of the diagonal and two rounds of joining (A 0; C B)^-1 = (A' 0; -B' C A' B'),
// on the fp32 matrix instruction.  G is summed in 64 bits and kept as two
// floats, so a difference of two large sums keeps its small decays.
//
// Blocks are independent, three workgroups a compute unit (bf16), and what bounds
// them is memory: bf16 [8, 2048], 20 heads of 128 with resets, 110 us for 194 MB
// read and 191 MB written; for the backward pass, which takes the transposed
// operands too, 200 us, 284 MB read and 460 MB written (a unit's wavefronts wait
// for loads 70% of the time).
#include "delta_tile.hpp"
#include "delta_ws.hpp"

namespace lrscan {
namespace delta {

// ---- blocks between resets ----
constexpr int kScanTokens = 16;  // of one thread

// Inclusive scan of one int a thread over the workgroup (max or sum).
template <bool MAX>
__device__ __forceinline__ int block_scan(int x, int* lds) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x = MAX ? max(x, y) : x + y;
    }
    __syncthreads();
    if (lane == 63) lds[w] = x;
    __syncthreads();
    for (int i = 0; i < w; ++i) x = MAX ? max(x, lds[i]) : x + lds[i];
    return x;
}

__global__ void __launch_bounds__(kScanThreads) delta_blocks(const uint8_t* reset, int T, int* starts, int* counts) {
    __shared__ int lds[kScanThreads / 64];
    __shared__ int carry[2];  // start of the segment that the tile begins in; blocks so far
    const int64_t b = blockIdx.x;
    reset += b * T;
    starts += b * ((int64_t)T + 1);
    if (threadIdx.x == 0) carry[0] = 0, carry[1] = 0;
    for (int64_t t0 = 0; t0 < T; t0 += kScanThreads * kScanTokens) {
        const int64_t mine = t0 + (int64_t)threadIdx.x * kScanTokens;
        uint32_t marks = 0;
        int latest = -1;
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j)
            if (mine + j < T && reset[mine + j]) marks |= 1u << j, latest = (int)(mine + j);
        const int upto = block_scan<true>(latest, lds);
        const int before = __shfl_up(upto, 1);
        __shared__ int edge[kScanThreads / 64];
        __syncthreads();
        if ((threadIdx.x & 63) == 63) edge[threadIdx.x >> 6] = upto;
        __syncthreads();
        int seg = (threadIdx.x & 63) ? before : threadIdx.x ? edge[(threadIdx.x >> 6) - 1] : -1;
        seg = max(seg, carry[0]);
        uint32_t first = 0;
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j) {
            if (mine + j >= T) break;
            if (marks >> j & 1) seg = (int)(mine + j);
            if (((mine + j) - seg) % kC == 0) first |= 1u << j;
        }
        const int n = __popc(first);
        const int total = block_scan<false>(n, lds);
        int at = carry[1] + total - n;
#pragma unroll
        for (int j = 0; j < kScanTokens; ++j)
            if (first >> j & 1) starts[at++] = (int)(mine + j) | (marks >> j & 1 ? kCut : 0);
        __syncthreads();
        if (threadIdx.x == kScanThreads - 1) {
            carry[0] = max(carry[0], upto);
            carry[1] += total;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        starts[carry[1]] = T;
        counts[b] = carry[1];
    }
}

constexpr int kS = kC + 4;  // floats of an LDS row

template <int DT, bool BWD>
__global__ void __launch_bounds__(kThreads, DT == DT_BF16 ? 3 : 2) delta_prep(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, int slots,
                                                       int width) {
    constexpr int NP = kPlanes<DT>;
    // 128 columns (fp32: 64) of K and Q at a time, then the block's matrices
    constexpr int kW = DT == DT_F32 ? 64 : 128, kKS = kW + 8, kPlane = kC * kKS;
    constexpr int kTile = 2 * NP * kPlane * 2, kMats = 3 * kC * kS * 4;
    __shared__ __attribute__((aligned(16))) char lds[kTile > kMats ? kTile : kMats];
    __shared__ float gh[kC], gl[kC], bt[kC];
    uint16_t* const tile = reinterpret_cast<uint16_t*>(lds);
    float* const N = reinterpret_cast<float*>(lds);
    float *const M = N + kC * kS, *const Ti = M + kC * kS;  // M: the outputs' weights, forward
    float* const tmp = Ti + 32;  // the inverse's upper right quarter, which nothing reads
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int64_t bh = scalar((int)blockIdx.x / slots), b = scalar((int)bh / s.H);
    const int h = scalar((int)bh % s.H), hk = scalar(h / (s.H / s.HK));
    const int n = blocks.count(b);
    // rows with more blocks than slots begin again at a slot of their own, so no XCD gets all of those
    for (int c = scalar((int)((blockIdx.x + bh) % slots)); c < n; c += slots) {
        int start, len;
        bool cut;
        blocks.at(b, c, start, len, cut);
        __syncthreads();  // the last block's LDS is read
        if (w == 0) {
            const bool ok = lane < len;
            // nothing enters a segment's first token that its decay could act on, so that decay is 1
            const bool first = lane == 0 && (cut || (start == 0 && !in.h0));
            float g = ok && !first ? *reinterpret_cast<const float*>(in.g.row(b, start + lane, h)) : 0.0f;
            g = g < -200.0f ? -200.0f : g;  // exp is 0 there in fp32; no infinity enters a difference
            const float beta = ok ? *reinterpret_cast<const float*>(in.beta.row(b, start + lane, h)) : 0.0f;
            double G = g;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const double y = __shfl_up(G, d);
                if (lane >= d) G += y;
            }
            const double end = __shfl(G, 63);
            const float hi = (float)G, lo = (float)(G - hi);
            gh[lane] = hi, gl[lane] = lo, bt[lane] = beta;
            if (ok) {
                const int64_t at = bh * s.T + start + lane;
                prep.gates[at] = f32x4{expf((float)G), expf((float)(end - G)), beta, hi};
                if (BWD) prep.gl[at] = lo;
            }
        }
        const Buffer krows = block_rows(in.k, b, hk, start, len), qrows = block_rows(in.q, b, hk, start, len);
        // K K^T and Q K^T: a wavefront's 16 rows against the tokens up to them
        f32x4 kk[4], qk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0, 0, 0, 0};
        for (int k0 = 0; k0 < s.K; k0 += kW) {
            Raw8<DT> ka[kW / 32], qa[kW / 32];
#pragma unroll
            for (int i = 0; i < kW / 32; ++i) {
                const int o = i * kThreads + threadIdx.x, r = o / (kW / 8), q = k0 + o % (kW / 8) * 8;
                ka[i].load(krows, r * (int)in.k.st, q, width);
                qa[i].load(qrows, r * (int)in.q.st, q, width);
            }
            if (k0) __syncthreads();
#pragma unroll
            for (int i = 0; i < kW / 32; ++i) {
                const int o = i * kThreads + threadIdx.x, at = o / (kW / 8) * kKS + o % (kW / 8) * 8;
                store_frag(tile + at, kPlane, ka[i].frag());
                store_frag(tile + NP * kPlane + at, kPlane, qa[i].frag());
            }
            __syncthreads();
#pragma unroll
            for (int ks = 0; ks < kW; ks += 32) {
                const Frag<NP> kf = row_frag<NP>(tile, kPlane, kKS, w * 16, ks, lane);
                const Frag<NP> qf = row_frag<NP>(tile + NP * kPlane, kPlane, kKS, w * 16, ks, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j <= w) {
                        const Frag<NP> bf = row_frag<NP>(tile, kPlane, kKS, j * 16, ks, lane);
                        mma(kk[j], kf, bf);
                        mma(qk[j], qf, bf);
                    }
            }
        }
        __syncthreads();  // the tiles are read
        for (int i = threadIdx.x; i < kC * kS; i += kThreads) Ti[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = j * 16 + ln;
            f32x4 back = {0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = w * 16 + lg * 4 + r;
                float m = 0.0f, a = 0.0f;
                if (j <= w && col <= i) {
                    const float d = expf((gh[i] - gh[col]) + (gl[i] - gl[col]));
                    a = d * qk[j][r];
                    m = col < i ? d * kk[j][r] : 0.0f;
                }
                N[i * kS + col] = m * bt[col];
                if (BWD) M[i * kS + col] = m;
                back[r] = a;
            }
            // rows (columns of the transposed ones) 0 .. 31 have nothing to read beyond (before) 32
            if (BWD) {
                if (col < len && (j < 2 || w >= 2))
                    store_planes(prep.att_t + ((bh * s.T + start + col) * 3) * kC + place(w * 16 + lg * 4), kC, back);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) M[(w * 16 + lg * 4 + r) * kS + col] = back[r];
            }
        }
        __syncthreads();

        // the inverse: 16x16 blocks of the diagonal, a column a lane
        {
            const float* D = N + (w * 16) * kS + w * 16;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float y = r == ln ? 1.0f : 0.0f;
#pragma unroll
                for (int q = 0; q < r; ++q) y = fmaf(-D[r * kS + q], x[q], y);
                x[r] = y;
            }
            if (lg == 0)
#pragma unroll
                for (int r = 0; r < 16; ++r) Ti[(w * 16 + r) * kS + w * 16 + ln] = x[r];
        }
        __syncthreads();
        // then of 32 and of 64
        const int r0 = (w >> 1) * 32;
        if (!(w & 1)) {
            const f32x4 y = mm16(N + (r0 + 16) * kS + r0, kS, Ti + r0 * kS + r0, kS, 16, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) tmp[(w * 8 + lg * 4 + r) * kS + ln] = y[r];
        }
        __syncthreads();
        if (!(w & 1)) {
            const f32x4 y = mm16(Ti + (r0 + 16) * kS + r0 + 16, kS, tmp + w * 8 * kS, kS, 16, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) Ti[(r0 + 16 + lg * 4 + r) * kS + r0 + ln] = -y[r];
        }
        __syncthreads();
        const int ta = (w >> 1) * 16, tb = (w & 1) * 16;
        {
            const f32x4 y = mm16(N + (32 + ta) * kS, kS, Ti + tb, kS, 32, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) tmp[(ta + lg * 4 + r) * kS + tb + ln] = y[r];
        }
        __syncthreads();
        {
            const f32x4 y = mm16(Ti + (32 + ta) * kS + 32, kS, tmp + tb, kS, 32, lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) Ti[(32 + ta + lg * 4 + r) * kS + tb + ln] = -y[r];
        }
        __syncthreads();

        // A product of 16 or 32 rows brings a value that is not finite to the rows before its
        // own too, as zero times it; what stands anywhere in the inverse stands in its last
        // row.  Then a column a lane, every row from those before it alone.
        if (__any(!(fabsf(Ti[(kC - 1) * kS + lane]) < INFINITY))) {
            __syncthreads();
            if (w == 0)
                for (int r = 0; r < kC; ++r) {
                    float y = r == lane ? 1.0f : 0.0f;
                    for (int q = 0; q < r; ++q) {
                        const float z = fmaf(-N[r * kS + q], Ti[q * kS + lane], y);
                        y = q >= lane ? z : y;  // the rows before the column's own are zeros
                    }
                    Ti[r * kS + lane] = y;
                    if (__any(!(fabsf(y) < INFINITY))) {  // then no row behind it is finite
                        for (int i = r + 1; i < kC; ++i) Ti[i * kS + lane] = lane <= i ? __builtin_nanf("") : 0.0f;
                        break;
                    }
                }
            __syncthreads();
        }

        // rows of the inverse and of the outputs' weights
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = i * kThreads + threadIdx.x, r = o >> 3, q = (o & 7) * 8;
            if (r < len && (r >= 32 || q < 32)) {
                // the eight elements that stand at q .. q + 7
                const int e = r * kS + (q & 32) + (q & 24) / 2;
                const int64_t to = (bh * s.T + start + r) * 3 * kC + q;
                store_frag(prep.inv + to, kC,
                           split8(*reinterpret_cast<const f32x4*>(Ti + e), *reinterpret_cast<const f32x4*>(Ti + e + 16)));
                if (!BWD)
                    store_frag(prep.att + to, kC,
                               split8(*reinterpret_cast<const f32x4*>(M + e), *reinterpret_cast<const f32x4*>(M + e + 16)));
            }
        }
        if (BWD) {
            // (I + diag(beta) M)^-1 = I - diag(beta) (I + N)^-1 M, its columns
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = j * 16 + ln;
                f32x4 y = {0, 0, 0, 0};
                if (j <= w) y = mm16(Ti + (w * 16) * kS + j * 16, kS, M + (j * 16) * kS + j * 16, kS, (w - j + 1) * 16, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = w * 16 + lg * 4 + r;
                    y[r] = (i == col ? 1.0f : 0.0f) - bt[i] * y[r];
                }
                if (col < len && (j < 2 || w >= 2))
                    store_planes(prep.inv_t + (bh * s.T + start + col) * 3 * kC + place(w * 16 + lg * 4), kC, y);
            }
        }
    }
}

hipError_t run_blocks(const DeltaShape& s, const uint8_t* reset, int* starts, int* counts, hipStream_t st) {
    delta_blocks<<<dim3((unsigned)s.B), dim3(kScanThreads), 0, st>>>(reset, (int)s.T, starts, counts);
    return hipGetLastError();
}

template <int DT, bool BWD>
hipError_t prep_of(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, hipStream_t st) {
    const int slots = (int)((s.T + kC - 1) / kC);
    delta_prep<DT, BWD><<<dim3((unsigned)(s.B * s.H * slots)), kThreads, 0, st>>>(s, in, blocks, prep, slots,
                                                                                   row_width(s.K, DT));
    return hipGetLastError();
}

hipError_t run_prep(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, bool backward,
                    hipStream_t st) {
    if (s.dtype == DT_F32)
        return backward ? prep_of<DT_F32, true>(s, in, blocks, prep, st) : prep_of<DT_F32, false>(s, in, blocks, prep, st);
    return backward ? prep_of<DT_BF16, true>(s, in, blocks, prep, st) : prep_of<DT_BF16, false>(s, in, blocks, prep, st);
}

}  // namespace delta
}  // namespace lrscan
