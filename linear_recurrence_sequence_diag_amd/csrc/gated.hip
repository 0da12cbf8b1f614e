// gated.hip -- the gated scan, one thread to V adjacent lanes of a batch row
// (the per-lane walk), its decode step, and the reduction of the decay
// gradient's partial sums.
//
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_i) x_t,
//   a_t = exp(-scale softplus(decay) sigmoid(gate_r))
//
// (mathematics and gradients in gated_math.hpp).  The transition and the input
// term are formed in registers from x and the two gate pre-activations, so a
// forward reads three arrays and writes one; formed by separate passes they
// would cost five more.  A reset step drops the state by a select, not by a
// product with 0, so an infinity or NaN in one segment does not reach the
// next.
//
// The walk is the form for sequences too short for tiles, for one decode step
// (T = 1) and for shapes past the tiles' index limits.  Memory bounds it, at
// two to four wavefronts a SIMD: bf16 [2048, 8, 2560] 78 us forward (336 MB,
// 4.3 TB/s) and 155 reverse (671 MB, 4.3 TB/s) on MI355X.
#include "column_sum.hpp"
#include "gated.hpp"
#include "gated_math.hpp"
#include "launch.hpp"
#include "quad.hpp"

namespace lrscan {

namespace {

constexpr int kBlock = 256;
// Rows of every operand loaded together, 2 for sequences of two.  Measured (us
// forward / reverse, bf16, 2 / 4 / 8 rows): [4096,2,1024] 28.8 / 43.2,
// 29.7 / 50.5, 35.5 / 79.5; [2048,8,2560] 77 / 154, 81 / 149, 79 / 212;
// [1024,16,2560] 74 / 155, 79 / 149, 71 / 209: 8 leave the reverse walk one
// wavefront a SIMD.
constexpr int kRowsAhead = 4;

// Non-temporal, as every row is read once.
template <int DT, bool ALIGNED>
__device__ __forceinline__ RowVec<DT> load_at(const char* row, int64_t d0, int nvalid) {
    return load_vec<DT, ALIGNED, true>(row + (size_t)d0 * Elem<DT>::bytes, 0, nvalid, 0.0f);
}

struct WalkArgs {
    GatedShape s;
    int64_t vpr;   // vectors of V lanes in a row
    int64_t rows;  // batch rows a thread walks, one after the other
};

// U rows are loaded ahead of the arithmetic.
template <int DT, bool ALIGNED, int U>
__global__ __launch_bounds__(kBlock) void gated_walk_fwd_kernel(GatedFwd p, WalkArgs w) {
    constexpr int V = Elem<DT>::V;
    const int64_t B = w.s.B, T = w.s.T, D = w.s.D;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t group = gid / w.vpr;
    if (group * w.rows >= B) return;
    const int64_t d0 = (gid - group * w.vpr) * V;
    const int nvalid = (int)((D - d0) < V ? (D - d0) : V);

    float rate[V], h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rate[j] = j < nvalid ? gate_rate(p.decay[d0 + j], p.scale) : 0.0f;
    const int64_t end = (group + 1) * w.rows < B ? (group + 1) * w.rows : B;
    for (int64_t bi = group * w.rows; bi < end; ++bi) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = (p.h0 && j < nvalid) ? p.h0[bi * D + d0 + j] : 0.0f;
        for (int64_t t0 = 0; t0 < T; t0 += U) {
            RowVec<DT> x[U], gr[U], gi[U];
            bool start[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = t0 + u < T ? t0 + u : T - 1;
                x[u] = load_at<DT, ALIGNED>(p.x.row(bi, t), d0, nvalid);
                gr[u] = load_at<DT, ALIGNED>(p.gr.row(bi, t), d0, nvalid);
                gi[u] = load_at<DT, ALIGNED>(p.gi.row(bi, t), d0, nvalid);
                start[u] = p.reset && p.reset[bi * T + t];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t0 + u < T) {
                    RowOut<DT> o;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const GatedStep g = gated_step_of(x[u].get(j), gr[u].get(j), gi[u].get(j), rate[j]);
                        const GatedStep f = gated_start_of(x[u].get(j), gi[u].get(j));
                        h[j] = start[u] ? f.b : fmaf(g.a, h[j], g.b);
                        o.v[j] = h[j];
                    }
                    if (p.out) store_row<DT, ALIGNED>(p.out, (size_t)((bi * T + t0 + u) * D + d0), nvalid, o);
                }
            }
        }
        if (p.last) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < nvalid) p.last[bi * D + d0 + j] = h[j];
        }
    }
}

// One step (T = 1): four channels of R batch rows to a thread, all their loads
// before the arithmetic; h0 may be last itself.  A decode step is one round of
// loads and stores long: 3.1 us at bf16 [32, 2560], whose 1.4 MB are 0.3.  A
// channel's rate costs about as much as a step, so R rows share it where rows
// are many.
template <int DT, bool FULL, int R>
__global__ __launch_bounds__(kBlock) void gated_step_kernel(GatedFwd p, int64_t B, int64_t D, uint32_t vpr) {
    constexpr int S = Elem<DT>::bytes;
    const uint32_t vec = blockIdx.x * blockDim.x + threadIdx.x;
    if (vec >= vpr) return;
    const int64_t d0 = (int64_t)vec * kQuad, b0 = (int64_t)blockIdx.y * R;
    const int nvalid = (int)((D - d0) < kQuad ? (D - d0) : kQuad);
    const size_t lo = (size_t)d0 * S;
    Quad<DT> x[R], gr[R], gi[R];
    Quad<DT_F32> h[R];
    bool start[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t b = b0 + r < B ? b0 + r : B - 1;
        x[r] = Quad<DT>::template load<FULL>(p.x.row(b, 0) + lo, nvalid);
        gr[r] = Quad<DT>::template load<FULL>(p.gr.row(b, 0) + lo, nvalid);
        gi[r] = Quad<DT>::template load<FULL>(p.gi.row(b, 0) + lo, nvalid);
        h[r] = p.h0 ? Quad<DT_F32>::template load<FULL>(reinterpret_cast<const char*>(p.h0 + b * D + d0), nvalid)
                    : Quad<DT_F32>::zero();
        start[r] = p.reset && p.reset[b];
    }
    const Quad<DT_F32> dc = Quad<DT_F32>::template load<FULL>(reinterpret_cast<const char*>(p.decay + d0), nvalid);
    float rate[kQuad];
#pragma unroll
    for (int j = 0; j < kQuad; ++j) rate[j] = gate_rate(dc.get(j), p.scale);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (b0 + r >= B) break;
        float v[kQuad];
#pragma unroll
        for (int j = 0; j < kQuad; ++j) {
            const GatedStep g = gated_step_of(x[r].get(j), gr[r].get(j), gi[r].get(j), rate[j]);
            const GatedStep f = gated_start_of(x[r].get(j), gi[r].get(j));
            v[j] = start[r] ? f.b : fmaf(g.a, h[r].get(j), g.b);
        }
        if (p.out) {
            Quad<DT> o;
            o.set(v);
            o.template store<FULL>(static_cast<char*>(p.out) + (size_t)(b0 + r) * D * S + lo, nvalid);
        }
        if (p.last) {
            Quad<DT_F32> o;
            o.set(v);
            o.template store<FULL>(reinterpret_cast<char*>(p.last + (b0 + r) * D + d0), nvalid);
        }
    }
}

// Compensated running sum (Neumaier): a channel's decay gradient may run over
// millions of steps in one thread.
struct Compensated {
    float s = 0.0f, c = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float t = s + x;
        c += fabsf(s) >= fabsf(x) ? (s - t) + x : (x - t) + s;
        s = t;
    }
};

template <int DT, bool ALIGNED, int U>
__global__ __launch_bounds__(kBlock) void gated_walk_bwd_kernel(GatedBwd p, WalkArgs w, float* part) {
    constexpr int V = Elem<DT>::V;
    const int64_t B = w.s.B, T = w.s.T, D = w.s.D;
    const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t group = gid / w.vpr;
    if (group * w.rows >= B) return;
    const int64_t d0 = (gid - group * w.vpr) * V;
    const int nvalid = (int)((D - d0) < V ? (D - d0) : V);

    float rate[V], carry[V];
    Compensated sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rate[j] = j < nvalid ? gate_rate(p.decay[d0 + j], p.scale) : 0.0f;
    const int64_t end = (group + 1) * w.rows < B ? (group + 1) * w.rows : B;
    for (int64_t bi = group * w.rows; bi < end; ++bi) {
#pragma unroll
        for (int j = 0; j < V; ++j) carry[j] = (p.grad_last && j < nvalid) ? p.grad_last[bi * D + d0 + j] : 0.0f;
        for (int64_t t1 = T; t1 > 0; t1 -= U) {  // rows t1 - 1, ..., t1 - U
            RowVec<DT> x[U], gr[U], gi[U], g[U], hp[U];
            bool start[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = t1 - 1 - u >= 0 ? t1 - 1 - u : 0;
                const int64_t tp = t > 0 ? t - 1 : 0;
                x[u] = load_at<DT, ALIGNED>(p.x.row(bi, t), d0, nvalid);
                gr[u] = load_at<DT, ALIGNED>(p.gr.row(bi, t), d0, nvalid);
                gi[u] = load_at<DT, ALIGNED>(p.gi.row(bi, t), d0, nvalid);
                g[u] = load_at<DT, ALIGNED>(static_cast<const char*>(p.g) + (size_t)((bi * T + t) * D) * Elem<DT>::bytes, d0,
                                            nvalid);
                hp[u] = load_at<DT, ALIGNED>(static_cast<const char*>(p.out) + (size_t)((bi * T + tp) * D) * Elem<DT>::bytes, d0,
                                             nvalid);
                start[u] = p.reset && p.reset[bi * T + t];
            }
            float block_sum[V];
#pragma unroll
            for (int j = 0; j < V; ++j) block_sum[j] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t t = t1 - 1 - u;
                if (t >= 0) {
                    RowOut<DT> ox, orr, oi;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float prev = hp[u].get(j);
                        if (t == 0) prev = (p.h0 && j < nvalid) ? p.h0[bi * D + d0 + j] : 0.0f;
                        const float lam = carry[j] + g[u].get(j);
                        const float xv = x[u].get(j), rv = gr[u].get(j), iv = gi[u].get(j);
                        const GatedGrad q = start[u] ? gated_start_grad_of(xv, iv, lam)
                                                     : gated_grad_of(xv, rv, iv, rate[j], prev, lam);
                        carry[j] = start[u] ? 0.0f : q.a * lam;
                        ox.v[j] = q.dx;
                        orr.v[j] = q.dgr;
                        oi.v[j] = q.dgi;
                        block_sum[j] += q.p;
                    }
                    store_row<DT, ALIGNED>(p.gx.row(bi, t), (size_t)d0, nvalid, ox);
                    store_row<DT, ALIGNED>(p.ggr.row(bi, t), (size_t)d0, nvalid, orr);
                    store_row<DT, ALIGNED>(p.ggi.row(bi, t), (size_t)d0, nvalid, oi);
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j].add(block_sum[j]);
        }
        if (p.grad_h0) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < nvalid) p.grad_h0[bi * D + d0 + j] = carry[j];
        }
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < nvalid) part[group * D + d0 + j] = sum[j].s + sum[j].c;
    }
}

template <int DT>
dim3 walk_grid(const GatedShape& s, int block, WalkArgs* w) {
    w->s = s;
    w->vpr = (s.D + Elem<DT>::V - 1) / Elem<DT>::V;
    w->rows = gated_walk_rows(s);
    const int64_t groups = (s.B + w->rows - 1) / w->rows;
    return dim3((unsigned)((groups * w->vpr + block - 1) / block));
}

template <int DT>
hipError_t walk_fwd_t(const GatedShape& s, const GatedFwd& p, hipStream_t st) {
    WalkArgs w;
    const dim3 grid = walk_grid<DT>(s, kBlock, &w);
    const bool al = gated_fwd_aligned(s, p);
    if (s.T <= 2) {
        if (al) hipLaunchKernelGGL((gated_walk_fwd_kernel<DT, true, 2>), grid, dim3(kBlock), 0, st, p, w);
        else hipLaunchKernelGGL((gated_walk_fwd_kernel<DT, false, 2>), grid, dim3(kBlock), 0, st, p, w);
    } else {
        if (al) hipLaunchKernelGGL((gated_walk_fwd_kernel<DT, true, kRowsAhead>), grid, dim3(kBlock), 0, st, p, w);
        else hipLaunchKernelGGL((gated_walk_fwd_kernel<DT, false, kRowsAhead>), grid, dim3(kBlock), 0, st, p, w);
    }
    return hipGetLastError();
}

// Workgroups of one wavefront spread a small batch over the CUs; rows are
// shared by fours once that leaves eight wavefronts to a CU.
template <int DT, bool FULL>
hipError_t step_t(const GatedShape& s, const GatedFwd& p, hipStream_t st) {
    const uint32_t vpr = (uint32_t)((s.D + kQuad - 1) / kQuad);
    const unsigned gx = (vpr + kWave - 1) / kWave;
    if ((int64_t)gx * s.B >= 4 * 2048)
        hipLaunchKernelGGL((gated_step_kernel<DT, FULL, 4>), dim3(gx, (unsigned)((s.B + 3) / 4)), dim3(kWave), 0, st,
                           p, s.B, s.D, vpr);
    else
        hipLaunchKernelGGL((gated_step_kernel<DT, FULL, 1>), dim3(gx, (unsigned)s.B), dim3(kWave), 0, st, p, s.B, s.D,
                           vpr);
    return hipGetLastError();
}

template <int DT>
hipError_t walk_bwd_t(const GatedShape& s, const GatedBwd& p, float* part, hipStream_t st) {
    WalkArgs w;
    const dim3 grid = walk_grid<DT>(s, kBlock, &w);
    const bool al = gated_bwd_aligned(s, p);
    if (s.T <= 2) {
        if (al) hipLaunchKernelGGL((gated_walk_bwd_kernel<DT, true, 2>), grid, dim3(kBlock), 0, st, p, w, part);
        else hipLaunchKernelGGL((gated_walk_bwd_kernel<DT, false, 2>), grid, dim3(kBlock), 0, st, p, w, part);
    } else {
        if (al) hipLaunchKernelGGL((gated_walk_bwd_kernel<DT, true, kRowsAhead>), grid, dim3(kBlock), 0, st, p, w, part);
        else hipLaunchKernelGGL((gated_walk_bwd_kernel<DT, false, kRowsAhead>), grid, dim3(kBlock), 0, st, p, w, part);
    }
    return hipGetLastError();
}

// grad_decay = slope(decay) * sum of the partial rows (of P / ln 2).
struct WriteDecay {
    const float* decay;
    float* grad;
    __device__ __forceinline__ void put(int64_t, int64_t c, float sum) const {
        grad[c] = decay_slope(decay[c]) * (kLn2 * sum);
    }
};

}  // namespace

bool operand_aligned(int64_t B, int64_t T, const Rows& r) {
    if (reinterpret_cast<uintptr_t>(r.p) % 16 != 0) return false;
    return (T == 1 || r.st % 16 == 0) && (B == 1 || r.sb % 16 == 0);
}

bool gated_fwd_aligned(const GatedShape& s, const GatedFwd& p) {
    const Shape c{s.B, s.T, s.D, s.dtype};
    const void* ptrs[1] = {p.out};
    return rows_aligned(c, ptrs, 1) && operand_aligned(s.B, s.T, p.x) && operand_aligned(s.B, s.T, p.gr) &&
           operand_aligned(s.B, s.T, p.gi);
}

bool gated_bwd_aligned(const GatedShape& s, const GatedBwd& p) {
    const Shape c{s.B, s.T, s.D, s.dtype};
    const void* ptrs[2] = {p.out, p.g};
    return rows_aligned(c, ptrs, 2) && operand_aligned(s.B, s.T, p.x) && operand_aligned(s.B, s.T, p.gr) &&
           operand_aligned(s.B, s.T, p.gi) && operand_aligned(s.B, s.T, p.gx) && operand_aligned(s.B, s.T, p.ggr) &&
           operand_aligned(s.B, s.T, p.ggi);
}

// A channel's rate costs a thread about as much as two steps, so short
// sequences share it (and one partial row of the decay gradient) among up to
// 16 steps' worth of batch rows, as long as that leaves eight wavefronts to
// a CU.  Measured on MI355X (us forward / reverse; one row to a thread, up to 8,
// 16 and 32 steps' worth):
//   bf16 [8192,2,1024]  53 /  94    44 /  74    48 /  63    49 /  63
//        [4096,4,1024]  39 /  82    38 /  77    37 /  67    37 /  67
//        [2048,8,2560]  75 / 155    75 / 155    82 / 149    78 / 167
//   f32  [2048,8,2560] 120 / 246   121 / 246   130 / 256   140 / 265
// (half as many wavefronts to a CU: [1024,4,1024] 15 / 29 for 13 / 27; twice as
// many: [4096,4,1024] 38 / 76 for 37 / 67).
int64_t gated_walk_rows(const GatedShape& s) {
    const int64_t v = s.dtype == DT_F32 ? Elem<DT_F32>::V : Elem<DT_BF16>::V;
    const int64_t threads = s.B * ((s.D + v - 1) / v);
    int64_t rows = 1;
    while (rows * 2 * s.T <= 16 && threads / (rows * 2) >= ((int64_t)1 << 17)) rows *= 2;
    return rows;
}

bool gated_walk_fits(const GatedShape& s) {
    const int64_t v = s.dtype == DT_F32 ? Elem<DT_F32>::V : Elem<DT_BF16>::V;
    return s.B * ((s.D + v - 1) / v) < ((int64_t)1 << 32) - kBlock;  // work-items of the grid
}

hipError_t launch_gated_walk_fwd(const GatedShape& s, const GatedFwd& p, hipStream_t st) {
    if (s.T == 1 && s.B <= 65535 && s.D < ((int64_t)1 << 31)) {
        const bool full = s.D % kQuad == 0;
        if (s.dtype == DT_F32) return full ? step_t<DT_F32, true>(s, p, st) : step_t<DT_F32, false>(s, p, st);
        return full ? step_t<DT_BF16, true>(s, p, st) : step_t<DT_BF16, false>(s, p, st);
    }
    return s.dtype == DT_F32 ? walk_fwd_t<DT_F32>(s, p, st) : walk_fwd_t<DT_BF16>(s, p, st);
}

hipError_t launch_gated_walk_bwd(const GatedShape& s, const GatedBwd& p, float* part, hipStream_t st) {
    return s.dtype == DT_F32 ? walk_bwd_t<DT_F32>(s, p, part, st) : walk_bwd_t<DT_BF16>(s, p, part, st);
}

bool gated_decay_fits(int64_t D) { return column_sum_fits(D); }

size_t gated_decay_scratch(int64_t rows, int64_t D) { return column_sum_scratch(rows, D); }

hipError_t launch_gated_decay(const float* part, int64_t rows, int64_t D, float* scratch,
                              const float* decay, float* grad_decay, hipStream_t st) {
    return launch_column_sum(part, rows, D, scratch, WriteDecay{decay, grad_decay}, st);
}

}  // namespace lrscan
