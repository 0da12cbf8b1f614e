// conv.hip -- the short causal convolution over tokens, one filter of K taps
// for each channel, with an optional sigmoid-weighted activation:
//
//   z_t = bias + sum_j w[j] x_{t-K+1+j},     y_t = z_t  or  z_t sigmoid(z_t)
//   gz_t = g_t dy/dz,   dx_s = sum_back w[K-1-back] gz_{s+back},
//   dw[j] = sum_t gz_t x_{t-K+1+j},   dbias = sum_t gz_t
//
// Inputs before the first come from `state` (the K - 1 inputs before it) or are
// zero, and a tap that would reach across a reset counts as zero.
//
// A thread owns V adjacent channels (16 bytes) of a chunk of consecutive
// tokens.  The last K - 1 inputs stay in registers, so a chunk re-reads only
// K - 1 rows of its neighbour; a reset clears them, which drops an infinity or
// NaN of the segment before.  The backward walks the chunk in the same order,
// recomputes z, and keeps the K - 1 input gradients that still wait for later
// gz in registers.  The parameter gradients are summed over the chunk in
// registers, over a workgroup's chunks through LDS, and over workgroups by
// column_sum, each in a fixed order.
#include "conv.hpp"

#include "column_sum.hpp"
#include "gated_math.hpp"
#include "launch.hpp"

namespace lrscan {

namespace {

constexpr int kBlock = 256;
constexpr int kFwdRows = 16;  // tokens of a chunk
constexpr int kBwdRows = 32;

// Workgroup blockIdx.x covers lane block blockIdx.x % ncb and `groups`
// consecutive chunks (a chunk: `rows` tokens of one batch row).
struct ConvGrid {
    uint32_t tpr;      // threads along a row (a power of two, at most 64)
    uint32_t groups;   // kBlock / tpr chunks side by side
    uint32_t vpr;      // vectors in a row
    uint32_t ncb;      // lane blocks
    uint32_t nchunks;  // chunks of a batch row
    uint32_t chunks;   // B * nchunks
    uint32_t blocks;   // workgroups along the chunks
    int rows;
};

int64_t chunks_of(const ConvShape& s, int rows) { return s.B * ((s.T + rows - 1) / rows); }

ConvGrid conv_grid(const ConvShape& s, int rows) {
    const int v = s.dtype == DT_F32 ? Elem<DT_F32>::V : Elem<DT_BF16>::V;
    ConvGrid g;
    g.rows = rows;
    g.vpr = (uint32_t)((s.D + v - 1) / v);
    g.tpr = 1;
    while (g.tpr < 64 && g.tpr < g.vpr) g.tpr *= 2;
    g.groups = kBlock / g.tpr;
    g.ncb = (g.vpr + g.tpr - 1) / g.tpr;
    g.nchunks = (uint32_t)((s.T + rows - 1) / rows);
    g.chunks = (uint32_t)chunks_of(s, rows);
    g.blocks = (g.chunks + g.groups - 1) / g.groups;
    return g;
}

struct ConvPos {
    int64_t bi, t0, t1, d0;  // batch row, tokens [t0, t1), first channel
    int nvalid;              // channels of the vector that exist; 0: an idle thread
};

template <int V>
__device__ __forceinline__ ConvPos conv_pos(const ConvGrid& g, int64_t T, int64_t D) {
    const uint32_t cb = blockIdx.x % g.ncb, rb = blockIdx.x / g.ncb;
    const uint32_t lane = threadIdx.x & (g.tpr - 1), grp = threadIdx.x / g.tpr;
    const uint32_t chunk = rb * g.groups + grp, vec = cb * g.tpr + lane;
    ConvPos p;
    p.nvalid = 0;
    p.bi = p.t0 = p.t1 = p.d0 = 0;
    if (chunk >= g.chunks || vec >= g.vpr) return p;
    const uint32_t b = chunk / g.nchunks;
    p.bi = b;
    p.t0 = (int64_t)(chunk - b * g.nchunks) * g.rows;
    p.t1 = p.t0 + g.rows < T ? p.t0 + g.rows : T;
    p.d0 = (int64_t)vec * V;
    p.nvalid = (int)((D - p.d0) < V ? (D - p.d0) : V);
    return p;
}

// The K - 1 inputs before token t0, oldest first, those of an earlier segment
// cleared.
template <int DT, bool ALIGNED, int K>
__device__ __forceinline__ void conv_warm(RowVec<DT> (&win)[K - 1], const Rows& x, const void* state,
                                          const uint8_t* reset, const ConvPos& p, int64_t T, int64_t D) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t t = p.t0 - (K - 1) + j;
        if (t >= 0)
            win[j] = load_row<DT, ALIGNED>(x.row(p.bi, t), (size_t)p.d0, p.nvalid, 0.0f);
        else if (state)
            win[j] = load_row<DT, ALIGNED>(state, (size_t)((p.bi * (K - 1) + t + K - 1) * D + p.d0),
                                           p.nvalid, 0.0f);
        else
            win[j] = RowVec<DT>::splat(0.0f);
        if (reset && t >= 0 && reset[p.bi * T + t]) {
#pragma unroll
            for (int i = 0; i < j; ++i) win[i] = RowVec<DT>::splat(0.0f);
        }
    }
}

template <int DT, int K>
__device__ __forceinline__ void conv_push(RowVec<DT> (&win)[K - 1], const RowVec<DT>& x) {
#pragma unroll
    for (int j = 0; j + 1 < K - 1; ++j) win[j] = win[j + 1];
    win[K - 2] = x;
}

template <int V, int K>
struct Taps {
    float w[K][V], bias[V];
    __device__ __forceinline__ void load(const float* wp, const float* bp, const ConvPos& p, int64_t D) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][j] = j < p.nvalid ? wp[k * D + p.d0 + j] : 0.0f;
            bias[j] = (bp && j < p.nvalid) ? bp[p.d0 + j] : 0.0f;
        }
    }
    template <int DT>
    __device__ __forceinline__ float z(const RowVec<DT> (&win)[K - 1], const RowVec<DT>& x, int j) const {
        float z = bias[j];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) z = fmaf(w[k][j], win[k].get(j), z);
        return fmaf(w[K - 1][j], x.get(j), z);
    }
};

template <int DT, bool ALIGNED, int K, bool SILU>
__global__ __launch_bounds__(kBlock) void conv_fwd_kernel(ConvFwd a, ConvGrid g, int64_t T, int64_t D) {
    constexpr int V = Elem<DT>::V, U = 4;
    const ConvPos p = conv_pos<V>(g, T, D);
    if (p.nvalid == 0) return;
    Taps<V, K> tp;
    tp.load(a.w, a.bias, p, D);
    RowVec<DT> win[K - 1];
    conv_warm<DT, ALIGNED, K>(win, a.x, a.state, a.reset, p, T, D);
    for (int64_t t = p.t0; t < p.t1; t += U) {
        RowVec<DT> x[U];
        bool start[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t tu = t + u < p.t1 ? t + u : p.t1 - 1;
            x[u] = load_row<DT, ALIGNED>(a.x.row(p.bi, tu), (size_t)p.d0, p.nvalid, 0.0f);
            start[u] = a.reset && a.reset[p.bi * T + tu];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u < p.t1) {
                if (start[u]) {
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) win[j] = RowVec<DT>::splat(0.0f);
                }
                RowOut<DT> o;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float z = tp.z(win, x[u], j);
                    o.v[j] = SILU ? z * sigmoid_f(z) : z;
                }
                store_row<DT, ALIGNED>(a.out, (size_t)((p.bi * T + t + u) * D + p.d0), p.nvalid, o);
                conv_push<DT, K>(win, x[u]);
            }
        }
    }
    if (a.last && p.t1 == T) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            RowOut<DT> o;
#pragma unroll
            for (int v = 0; v < V; ++v) o.v[v] = win[j].get(v);
            store_row<DT, ALIGNED>(a.last, (size_t)((p.bi * (K - 1) + j) * D + p.d0), p.nvalid, o);
        }
    }
}

template <int DT, bool ALIGNED, int K, bool SILU>
__global__ __launch_bounds__(kBlock) void conv_bwd_kernel(ConvBwd a, ConvGrid g, int64_t T, int64_t D,
                                                          float* part) {
    constexpr int V = Elem<DT>::V, U = 4;
    __shared__ float s_part[kBlock * V];
    const ConvPos p = conv_pos<V>(g, T, D);
    float dw[K][V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        db[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][j] = 0.0f;
    }
    if (p.nvalid > 0) {
        Taps<V, K> tp;
        tp.load(a.w, a.bias, p, D);
        RowVec<DT> win[K - 1];
        conv_warm<DT, ALIGNED, K>(win, a.x, a.state, a.reset, p, T, D);
        float acc[K - 1][V];  // input gradients of tokens t - K + 1 .. t - 1
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
        int age = K - 1;  // tokens back that still lie in the segment (capped)
        const int64_t end = p.t0 + g.rows;  // one past the chunk's last token, which may lie past T
        for (int64_t t = p.t0; t < end + K - 1; t += U) {
            RowVec<DT> x[U], gr[U];
            bool start[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t tu = t + u < T ? t + u : T - 1;
                x[u] = load_row<DT, ALIGNED>(a.x.row(p.bi, tu), (size_t)p.d0, p.nvalid, 0.0f);
                gr[u] = load_row<DT, ALIGNED>(a.g, (size_t)((p.bi * T + tu) * D + p.d0), p.nvalid, 0.0f);
                start[u] = a.reset && a.reset[p.bi * T + tu];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t tu = t + u, s = tu - (K - 1);
                if (tu >= end + K - 1) break;
                const bool live = tu < T;
                if (live) {
                    age = start[u] ? 0 : (age < K - 1 ? age + 1 : K - 1);
                    if (start[u]) {
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) win[j] = RowVec<DT>::splat(0.0f);
                    }
                }
                RowOut<DT> o;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float gz = 0.0f;
                    if (live) {
                        gz = gr[u].get(j);
                        if constexpr (SILU) {
                            const float z = tp.z(win, x[u], j);
                            const Sigmoid q = sigmoid_pair(z);
                            gz *= q.s * fmaf(z, q.c, 1.0f);
                        }
                        if (tu < end) {
                            db[j] += gz;
                            dw[K - 1][j] = fmaf(gz, x[u].get(j), dw[K - 1][j]);
#pragma unroll
                            for (int k = 0; k < K - 1; ++k) dw[k][j] = fmaf(gz, win[k].get(j), dw[k][j]);
                        }
#pragma unroll
                        for (int i = 0; i < K - 1; ++i)
                            if (K - 1 - i <= age) acc[i][j] = fmaf(tp.w[i][j], gz, acc[i][j]);
                    }
                    o.v[j] = acc[0][j];
#pragma unroll
                    for (int i = 0; i + 1 < K - 1; ++i) acc[i][j] = acc[i + 1][j];
                    acc[K - 2][j] = tp.w[K - 1][j] * gz;
                }
                if (live) conv_push<DT, K>(win, x[u]);
                // token s is complete: it is the chunk's, or one of the state's
                if (s < T && (s >= p.t0 || (s < 0 && p.t0 == 0 && a.grad_state))) {
                    const int64_t back = T - 1 - s;  // its place in `last`, from the end
                    if (a.grad_last && back < K - 1 && back <= age) {
                        const RowVec<DT> gl = load_row<DT, ALIGNED>(
                            a.grad_last, (size_t)((p.bi * (K - 1) + K - 2 - back) * D + p.d0), p.nvalid, 0.0f);
#pragma unroll
                        for (int j = 0; j < V; ++j) o.v[j] += gl.get(j);
                    }
                    if (s >= 0)
                        store_row<DT, ALIGNED>(a.gx.row(p.bi, s), (size_t)p.d0, p.nvalid, o);
                    else
                        store_row<DT, ALIGNED>(a.grad_state,
                                               (size_t)((p.bi * (K - 1) + s + K - 1) * D + p.d0), p.nvalid, o);
                }
            }
        }
    }
    if (!part) return;
    // the workgroup's chunks, tap by tap (the bias last)
    const uint32_t cb = blockIdx.x % g.ncb, rb = blockIdx.x / g.ncb;
    const uint32_t width = g.tpr * V;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) s_part[threadIdx.x * V + j] = k < K ? dw[k < K ? k : 0][j] : db[j];
        __syncthreads();
        for (uint32_t e = threadIdx.x; e < width; e += kBlock) {
            const int64_t d = (int64_t)cb * width + e;
            if (d < D) {
                float t = 0.0f;
                for (uint32_t q = 0; q < g.groups; ++q) t += s_part[q * width + e];
                part[((size_t)rb * (K + 1) + k) * D + d] = t;
            }
        }
    }
}

// Column c of the partial rows: tap c / D of channel c % D, the bias as tap K.
struct WriteParams {
    float *w, *bias;
    int64_t nw;
    __device__ __forceinline__ void put(int64_t, int64_t c, float sum) const {
        if (c < nw) {
            if (w) w[c] = sum;
        } else if (bias) {
            bias[c - nw] = sum;
        }
    }
};

bool conv_aligned(const ConvShape& s, const void* const* ptrs, int n, const Rows* const* rows, int nr) {
    const Shape c{s.B, s.T, s.D, s.dtype};
    if (!rows_aligned(c, ptrs, n)) return false;
    for (int i = 0; i < nr; ++i)
        if (!operand_aligned(s.B, s.T, *rows[i])) return false;
    return true;
}

template <int DT, bool AL, int K>
void fwd_launch(const ConvShape& s, const ConvFwd& p, const ConvGrid& g, hipStream_t st) {
    const dim3 grid(g.ncb * g.blocks), block(kBlock);
    if (s.silu) hipLaunchKernelGGL((conv_fwd_kernel<DT, AL, K, true>), grid, block, 0, st, p, g, s.T, s.D);
    else hipLaunchKernelGGL((conv_fwd_kernel<DT, AL, K, false>), grid, block, 0, st, p, g, s.T, s.D);
}

template <int DT, bool AL, int K>
void bwd_launch(const ConvShape& s, const ConvBwd& p, const ConvGrid& g, float* part, hipStream_t st) {
    const dim3 grid(g.ncb * g.blocks), block(kBlock);
    if (s.silu)
        hipLaunchKernelGGL((conv_bwd_kernel<DT, AL, K, true>), grid, block, 0, st, p, g, s.T, s.D, part);
    else
        hipLaunchKernelGGL((conv_bwd_kernel<DT, AL, K, false>), grid, block, 0, st, p, g, s.T, s.D, part);
}

template <int DT, bool AL>
void fwd_taps(const ConvShape& s, const ConvFwd& p, const ConvGrid& g, hipStream_t st) {
    if (s.K == 2) fwd_launch<DT, AL, 2>(s, p, g, st);
    else if (s.K == 3) fwd_launch<DT, AL, 3>(s, p, g, st);
    else fwd_launch<DT, AL, 4>(s, p, g, st);
}

template <int DT, bool AL>
void bwd_taps(const ConvShape& s, const ConvBwd& p, const ConvGrid& g, float* part, hipStream_t st) {
    if (s.K == 2) bwd_launch<DT, AL, 2>(s, p, g, part, st);
    else if (s.K == 3) bwd_launch<DT, AL, 3>(s, p, g, part, st);
    else bwd_launch<DT, AL, 4>(s, p, g, part, st);
}

}  // namespace

bool conv_fits(const ConvShape& s) {
    if (s.D >= ((int64_t)1 << 31)) return false;
    for (const int rows : {kFwdRows, kBwdRows}) {
        const int64_t chunks = chunks_of(s, rows);
        if (chunks >= ((int64_t)1 << 31)) return false;
        const ConvGrid g = conv_grid(s, rows);
        // work-items of the grid in 32 bits
        if ((uint64_t)g.ncb * g.blocks >= ((uint64_t)1 << 32) / kBlock) return false;
    }
    return true;
}

size_t conv_part_bytes(const ConvShape& s) {
    return (size_t)conv_grid(s, kBwdRows).blocks * (size_t)(s.K + 1) * (size_t)s.D * 4;
}

size_t conv_sum_scratch(const ConvShape& s) {
    return column_sum_scratch(conv_grid(s, kBwdRows).blocks, (s.K + 1) * s.D);
}

hipError_t launch_conv_fwd(const ConvShape& s, const ConvFwd& p, hipStream_t st) {
    const ConvGrid g = conv_grid(s, kFwdRows);
    const void* ptrs[3] = {p.out, p.state, p.last};
    const Rows* rows[1] = {&p.x};
    const bool al = conv_aligned(s, ptrs, 3, rows, 1);
    if (s.dtype == DT_F32) al ? fwd_taps<DT_F32, true>(s, p, g, st) : fwd_taps<DT_F32, false>(s, p, g, st);
    else al ? fwd_taps<DT_BF16, true>(s, p, g, st) : fwd_taps<DT_BF16, false>(s, p, g, st);
    return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvShape& s, const ConvBwd& p, float* part, float* scratch,
                           float* grad_w, float* grad_bias, hipStream_t st) {
    const ConvGrid g = conv_grid(s, kBwdRows);
    const void* ptrs[4] = {p.state, p.g, p.grad_last, p.grad_state};
    const Rows* rows[2] = {&p.x, &p.gx};
    const bool al = conv_aligned(s, ptrs, 4, rows, 2);
    if (s.dtype == DT_F32)
        al ? bwd_taps<DT_F32, true>(s, p, g, part, st) : bwd_taps<DT_F32, false>(s, p, g, part, st);
    else
        al ? bwd_taps<DT_BF16, true>(s, p, g, part, st) : bwd_taps<DT_BF16, false>(s, p, g, part, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !part) return e;
    return launch_column_sum(part, (int64_t)g.blocks, (int64_t)(s.K + 1) * s.D, scratch,
                             WriteParams{grad_w, grad_bias, (int64_t)s.K * s.D}, st);
}

}  // namespace lrscan
