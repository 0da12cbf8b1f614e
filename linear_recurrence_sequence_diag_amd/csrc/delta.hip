// delta.hip -- gated delta rule: the passes of a call, and the step of one token.
//
// Forward: [blocks between resets], prep, walk.  Backward: the same with the
// entering states kept, the walk back, and the gradients block by block.
#include "delta_tile.hpp"
#include "delta_ws.hpp"

namespace lrscan {

using namespace delta;

namespace {

HeadRows contiguous(const DeltaShape& s, const void* p, int64_t heads, int width) {
    const int64_t sh = (int64_t)width * (s.dtype == DT_F32 ? 4 : 2);
    return HeadRows{static_cast<char*>(const_cast<void*>(p)), s.T * heads * sh, heads * sh, sh};
}

constexpr int kStepColumns = 64;  // of a workgroup of the step
int step_groups(const DeltaShape& s) { return (s.V + kStepColumns - 1) / kStepColumns; }

Copies copies(const DeltaShape& s, const DeltaIn& in, const void* grad_out) {
    const int e = s.dtype == DT_F32 ? 4 : 2;
    return Copies{!rows_whole(in.q, s.K, e), !rows_whole(in.k, s.K, e), !rows_whole(in.v, s.V, e),
                  grad_out && !rows_whole(contiguous(s, grad_out, s.H, s.V), s.V, e)};
}

}  // namespace

bool delta_fits(const DeltaShape& s, DeltaPass pass, bool reset) {
    if (s.K > kDeltaMaxK || s.V > 65536 || s.H > 65536 || s.T > ((int64_t)1 << 30)) return false;
    if ((int64_t)s.H * s.V > (1 << 22) || (int64_t)s.HK * s.K > (1 << 22)) return false;  // 32-bit offsets in a block's rows
    // work-items of a grid in 32 bits (B * T * H * V is within 2^40)
    auto grid_fits = [](int64_t workgroups, int64_t threads) { return workgroups < ((int64_t)1 << 32) / threads; };
    const int64_t slots = (s.T + kC - 1) / kC, heads = s.B * s.H;
    if (pass == kDeltaStep) return grid_fits(heads * step_groups(s), kThreads);
    // the walks (of few heads, which is where parts are formed and columns spread, they are far smaller)
    if (!grid_fits((heads + 7) / 8 * 8 * ((s.V + 127) / 128), kWalkThreads)) return false;
    if (reset && !grid_fits(s.B, kScanThreads)) return false;
    if (pass == kDeltaBackward && !grid_fits(s.B * s.HK * slots, kGradThreads)) return false;
    return grid_fits(heads * slots, kThreads);
}

size_t delta_ws_bytes(const DeltaShape& s, const DeltaIn* in, const void* grad_out, bool backward) {
    if (!in) return Layout(s, backward, true, Copies{true, true, true, true}).total;
    return Layout(s, backward, in->reset != nullptr, copies(s, *in, grad_out)).total;
}

namespace {

struct Pass {
    DeltaIn in;
    HeadRows go;
    Blocks blocks;
    Prep prep;
    Kept keep;
    Parts parts;
};

hipError_t begin(const DeltaShape& s, const DeltaIn& in, const void* grad_out, void* ws, hipStream_t st, Pass* pass) {
    const bool backward = grad_out != nullptr;
    const Copies copy = copies(s, in, grad_out);
    const Layout l(s, backward, in.reset != nullptr, copy);
    char* base = static_cast<char*>(ws);
    auto f = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
    auto planes = [&](size_t o) { return reinterpret_cast<uint16_t*>(base + o); };
    int* starts = in.reset ? reinterpret_cast<int*>(base + l.starts) : nullptr;
    int* counts = in.reset ? reinterpret_cast<int*>(base + l.counts) : nullptr;
    pass->in = in;
    pass->blocks = Blocks{starts, counts, (int)s.T};
    pass->prep = Prep{reinterpret_cast<f32x4*>(base + l.gates), f(l.gl), planes(l.inv), planes(l.att), planes(l.att_t),
                      planes(l.inv_t)};
    pass->keep = Kept{f(l.x), f(l.r), f(l.s), f(l.ds), reinterpret_cast<f32x4*>(base + l.sums)};
    pass->parts = Parts{sequence_parts(s), f(l.between), f(l.behind), f(l.map), backward ? f(l.map_t) : nullptr};
    RowCopies c{};
    auto whole = [&](HeadRows* rows, bool wanted, size_t o, int64_t heads, int n) {
        if (!wanted) return;
        const int width = row_width(n, s.dtype);
        c.of[c.count++] = RowCopies::One{*rows, base + o, heads, s.B * s.T * heads, n, width};
        *rows = contiguous(s, base + o, heads, width);
    };
    whole(&pass->in.q, copy.q, l.q, s.HK, s.K);
    whole(&pass->in.k, copy.k, l.k, s.HK, s.K);
    whole(&pass->in.v, copy.v, l.v, s.H, s.V);
    if (backward) {
        pass->go = contiguous(s, grad_out, s.H, s.V);
        whole(&pass->go, copy.go, l.go, s.H, s.V);
    }
    hipError_t e = run_copies(c, s.T, s.dtype, st);
    if (e == hipSuccess && in.reset) e = run_blocks(s, in.reset, starts, counts, st);
    if (e != hipSuccess) return e;
    return run_prep(s, pass->in, pass->blocks, pass->prep, backward, st);
}

}  // namespace

hipError_t launch_delta_fwd(const DeltaShape& s, const DeltaIn& in, const DeltaFwd& p, void* ws, hipStream_t st) {
    Pass pass;
    const hipError_t e = begin(s, in, nullptr, ws, st, &pass);
    if (e != hipSuccess) return e;
    return run_walk(s, pass.in, pass.blocks, pass.prep, p, nullptr, pass.parts, st);
}

hipError_t launch_delta_bwd(const DeltaShape& s, const DeltaIn& in, const DeltaBwd& p, void* ws, hipStream_t st) {
    Pass pass;
    hipError_t e = begin(s, in, p.grad_out, ws, st, &pass);
    if (e != hipSuccess) return e;
    e = run_walk(s, pass.in, pass.blocks, pass.prep, DeltaFwd{nullptr, nullptr}, &pass.keep, pass.parts, st);
    if (e != hipSuccess) return e;
    e = run_walk_back(s, pass.in, pass.blocks, pass.prep, p, pass.go, pass.keep, pass.parts, st);
    if (e != hipSuccess) return e;
    return run_grads(s, pass.in, pass.blocks, pass.prep, p, pass.go, pass.keep, st);
}

namespace delta {

// One launch for all operands, a wavefront for a row (fp32 [3, 777], 6 heads of 101
// and 2 of 70: 11 us, most of it latency, where three launches took 15).
template <class E>
__global__ void __launch_bounds__(kThreads) delta_copy(RowCopies copies, int64_t T) {
    const RowCopies::One c = copies.of[blockIdx.y];
    const int lane = threadIdx.x & 63;
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); r < c.rows; r += (int64_t)gridDim.x * (kThreads / 64)) {
        const int64_t bt = r / c.heads, b = bt / T;
        const E* from = reinterpret_cast<const E*>(c.from.row(b, bt - b * T, r - bt * c.heads));
        for (int x = lane; x < c.width; x += 64) static_cast<E*>(c.to)[r * c.width + x] = x < c.n ? from[x] : E(0);
    }
}

hipError_t run_copies(const RowCopies& c, int64_t T, int dtype, hipStream_t st) {
    if (c.count == 0) return hipSuccess;
    int64_t rows = 0;
    for (int i = 0; i < c.count; ++i) rows = c.of[i].rows > rows ? c.of[i].rows : rows;
    const int64_t blocks = (rows + kThreads / 64 - 1) / (kThreads / 64);
    const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048), (unsigned)c.count);
    if (dtype == DT_F32)
        delta_copy<uint32_t><<<grid, kThreads, 0, st>>>(c, T);
    else
        delta_copy<uint16_t><<<grid, kThreads, 0, st>>>(c, T);
    return hipGetLastError();
}

}  // namespace delta

// ---- one token ----
//
// S' = a S + k u^T with u = beta (v - a S^T k), o = scale S'^T q, of which
// S^T k, S^T q and q.k are sums over one pass of S: o = scale (a S^T q + (q.k) u).
// A workgroup has COLS columns of a head; its threads hold CV columns of every
// RG-th row in registers between the sums and the update.  Bytes of the state
// bound it (bf16, 32 rows of 20 heads of 128 by 128: 20.5 us for 84 MB, 4.1 TB/s;
// fp32, one row of 8 heads of 64 by 64: 6.1 us, a launch and one round of loads).
// Every thread writes the elements that it read, so the new state may replace the
// old one.
namespace delta {

template <int DT, int COLS, int CV>
__global__ void __launch_bounds__(kThreads) delta_step(DeltaShape s, DeltaIn in, DeltaFwd p, int groups) {
    constexpr int CG = COLS / CV, RG = kThreads / CG, ROWS = kDeltaMaxK / RG;
    __shared__ float qs[kDeltaMaxK], ks[kDeltaMaxK];
    __shared__ float sk[RG][COLS], sq[RG][COLS];
    __shared__ float dots[kThreads / 64];
    const int64_t bh = blockIdx.x / groups, b = bh / s.H;
    const int h = (int)(bh % s.H), hk = h / (s.H / s.HK);
    const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
    const int col = (int)(blockIdx.x % groups) * COLS + cg * CV;
    const float* state = in.reset && in.reset[b] ? nullptr : in.h0;
    typedef float vec __attribute__((ext_vector_type(CV)));
    vec S[ROWS];
    const int64_t base = bh * s.K * s.V + col;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int d = i * RG + rg;
        S[i] = vec(0.0f);
        if (state && d < s.K && col < s.V) S[i] = *reinterpret_cast<const vec*>(state + base + (int64_t)d * s.V);
    }
    float dot = 0.0f;
    {
        const int d = threadIdx.x;
        float q = 0.0f, k = 0.0f;
        if (d < s.K) q = load1<DT>(in.q.row(b, 0, hk), d), k = load1<DT>(in.k.row(b, 0, hk), d);
        qs[d] = q, ks[d] = k;
        dot = q * k;
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) dot += __shfl_xor(dot, m);
    if ((threadIdx.x & 63) == 0) dots[threadIdx.x >> 6] = dot;
    __syncthreads();
    vec a = vec(0.0f), q = vec(0.0f);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int d = i * RG + rg;
#pragma unroll
        for (int c = 0; c < CV; ++c) {
            a[c] = fmaf(ks[d], S[i][c], a[c]);
            q[c] = fmaf(qs[d], S[i][c], q[c]);
        }
    }
    *reinterpret_cast<vec*>(&sk[rg][cg * CV]) = a;
    *reinterpret_cast<vec*>(&sq[rg][cg * CV]) = q;
    __syncthreads();
    a = q = vec(0.0f);
    for (int r = 0; r < RG; ++r) {
        a += *reinterpret_cast<const vec*>(&sk[r][cg * CV]);
        if (p.out) q += *reinterpret_cast<const vec*>(&sq[r][cg * CV]);
    }
    if (col >= s.V) return;
    const float decay = expf(*reinterpret_cast<const float*>(in.g.row(b, 0, h)));
    const float beta = *reinterpret_cast<const float*>(in.beta.row(b, 0, h));
    const float qk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    vec u;
#pragma unroll
    for (int c = 0; c < CV; ++c) {
        const float v = load1<DT>(in.v.row(b, 0, h), col + c);
        // a state that a segment starts from is zero whatever the decay
        u[c] = beta * (state ? fmaf(-decay, a[c], v) : v);
        if (p.out && rg == 0) put1<DT>(p.out, bh * s.V + col + c, in.scale * (state ? fmaf(decay, q[c], qk * u[c]) : qk * u[c]));
    }
    if (p.last)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int d = i * RG + rg;
            if (d < s.K) {
                vec y;
#pragma unroll
                for (int c = 0; c < CV; ++c) y[c] = state ? fmaf(ks[d], u[c], decay * S[i][c]) : ks[d] * u[c];
                *reinterpret_cast<vec*>(p.last + base + (int64_t)d * s.V) = y;
            }
        }
}

template <int DT, int COLS, int CV>
hipError_t step(const DeltaShape& s, const DeltaIn& in, const DeltaFwd& p, hipStream_t st) {
    const int groups = step_groups(s);
    delta_step<DT, COLS, CV><<<dim3((unsigned)(s.B * s.H * groups)), kThreads, 0, st>>>(s, in, p, groups);
    return hipGetLastError();
}

template <int DT>
hipError_t step_of(const DeltaShape& s, const DeltaIn& in, const DeltaFwd& p, hipStream_t st) {
    const bool vec = (reinterpret_cast<uintptr_t>(in.h0) | reinterpret_cast<uintptr_t>(p.last) |
                      (uintptr_t)(s.V * 4)) % 16 == 0;
    if (!vec) return step<DT, kStepColumns, 1>(s, in, p, st);
    return step<DT, kStepColumns, 4>(s, in, p, st);
}

}  // namespace delta

hipError_t launch_delta_step(const DeltaShape& s, const DeltaIn& in, const DeltaFwd& p, hipStream_t st) {
    return s.dtype == DT_BF16 ? step_of<DT_BF16>(s, in, p, st) : step_of<DT_F32>(s, in, p, st);
}

}  // namespace lrscan
