// embed.hip -- the embedding lookup with scaling and its gradient by sorted
// tokens:
//
//   out[n] = scale W[ids[n]],     grad_W[v] = scale sum_{n: ids[n] = v} g[n]
//
// Ids outside [0, V) name no row: the lookup writes zeros for them and the
// gradient leaves them out.
//
// The gradient is a sum over tokens whose number for a row is anything from
// none to all of them, and its order has to be fixed for results to repeat.
// So the tokens are sorted by id first, stably, with their positions (a radix
// sort of digits of at most 10 bits, each pass one counting and one
// scattering launch), the first sorted place of every row is looked up, and
// each row then adds its own tokens' gradients in the order of their
// positions, in fp32, and is rounded and written once: zeros where it has no
// token.
#include "embed.hpp"

#include "device.hpp"
#include "launch.hpp"

namespace lrscan {

namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;
constexpr int kMaxDigitBits = 10;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int64_t kSortTile = 2048;      // tokens a workgroup sorts, at least
constexpr int64_t kMaxSortBlocks = 256;  // then a workgroup takes more

template <int IB>
__device__ __forceinline__ int64_t load_id(const void* ids, int64_t n) {
    if constexpr (IB == 8) return reinterpret_cast<const int64_t*>(ids)[n];
    else return reinterpret_cast<const int32_t*>(ids)[n];
}

// ---------------------------------------------------------------------------
// lookup: one thread to a 16-byte vector of an output row
// ---------------------------------------------------------------------------
template <int DT, int IB, bool ALIGNED>
__global__ __launch_bounds__(kBlock) void embed_fwd_kernel(const void* __restrict__ ids,
                                                           const void* __restrict__ w, float scale,
                                                           void* __restrict__ out, int64_t N,
                                                           int64_t rows, int64_t D, uint32_t vpr) {
    constexpr int V = Elem<DT>::V;
    // blockIdx.y counts groups of vectors of a row, so a wavefront stays in one row
    const uint32_t vec = blockIdx.y * kWave + threadIdx.x % kWave;
    const int64_t n = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    if (n >= N || vec >= vpr) return;
    const int64_t d0 = (int64_t)vec * V;
    const int nvalid = (int)((D - d0) < V ? (D - d0) : V);
    const int64_t id = load_id<IB>(ids, n);
    RowOut<DT> o;
    if (id >= 0 && id < rows) {
        const RowVec<DT> r = load_row<DT, ALIGNED>(w, (size_t)id * (size_t)D + (size_t)d0, nvalid, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = scale * r.get(j);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = 0.0f;
    }
    store_row<DT, ALIGNED>(out, (size_t)n * (size_t)D + (size_t)d0, nvalid, o);
}

// ---------------------------------------------------------------------------
// stable radix sort of (id, position)
// ---------------------------------------------------------------------------
struct SortPass {
    uint32_t N, tile, blocks;  // tokens; of one workgroup; workgroups
    int shift, bits;
};

// Where a pass reads its keys: the ids themselves (an id that names no row is
// the key V, after every row), or what the pass before wrote.
template <int IB>
struct KeysFromIds {
    const void* ids;
    int64_t V;
    __device__ __forceinline__ uint32_t key(uint32_t n) const {
        const int64_t id = load_id<IB>(ids, n);
        return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
    }
    __device__ __forceinline__ uint32_t pos(uint32_t n) const { return n; }
};
struct KeysFromPass {
    const uint32_t *keys, *poss;
    __device__ __forceinline__ uint32_t key(uint32_t n) const { return keys[n]; }
    __device__ __forceinline__ uint32_t pos(uint32_t n) const { return poss[n]; }
};

// counts[block][digit]: tokens of the workgroup's tile with that digit.
template <class Src>
__global__ __launch_bounds__(kBlock) void sort_count_kernel(Src src, SortPass p, uint32_t* counts) {
    __shared__ uint32_t s_n[kMaxDigits];
    const uint32_t digits = 1u << p.bits;
    for (uint32_t d = threadIdx.x; d < digits; d += kBlock) s_n[d] = 0;
    __syncthreads();
    const uint64_t n0 = (uint64_t)blockIdx.x * p.tile;
    const uint64_t n1 = n0 + p.tile < p.N ? n0 + p.tile : p.N;
    for (uint64_t n = n0 + threadIdx.x; n < n1; n += kBlock)
        atomicAdd(&s_n[(src.key((uint32_t)n) >> p.shift) & (digits - 1)], 1u);
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < digits; d += kBlock) counts[(size_t)blockIdx.x * digits + d] = s_n[d];
}

// Every token of the tile to its place: the tokens of smaller digits, those of
// its digit in earlier workgroups, in earlier wavefronts of its own, and
// before it in its wavefront.  A wavefront owns consecutive tokens and ranks
// 64 at a time by the lanes that hold the same digit.
template <class Src>
__global__ __launch_bounds__(kBlock) void sort_scatter_kernel(Src src, SortPass p, const uint32_t* counts,
                                                              uint32_t* keys, uint32_t* poss) {
    __shared__ uint32_t s_at[kWaves][kMaxDigits];  // next place of each digit, by wavefront
    __shared__ uint32_t s_scan[kBlock];
    const uint32_t digits = 1u << p.bits;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const uint64_t n0 = (uint64_t)blockIdx.x * p.tile;
    const uint64_t n1 = n0 + p.tile < p.N ? n0 + p.tile : p.N;
    // this wavefront's tokens
    const uint64_t w0 = n0 + (uint64_t)wave * (p.tile / kWaves);
    const uint64_t w1 = w0 + p.tile / kWaves < n1 ? w0 + p.tile / kWaves : n1;

    for (uint32_t d = tid; d < kWaves * kMaxDigits; d += kBlock) (&s_at[0][0])[d] = 0;
    __syncthreads();
    for (uint64_t n = w0 + lane; n < w1; n += kWave)
        atomicAdd(&s_at[wave][(src.key((uint32_t)n) >> p.shift) & (digits - 1)], 1u);

    // totals of this thread's digits, and what earlier workgroups hold of them
    constexpr int Q = kMaxDigits / kBlock;
    uint32_t total[Q], before[Q], mine = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const uint32_t d = tid * Q + q;
        total[q] = before[q] = 0;
        if (d < digits) {
            for (uint32_t b = 0; b < p.blocks; ++b) {
                const uint32_t c = counts[(size_t)b * digits + d];
                if (b < blockIdx.x) before[q] += c;
                total[q] += c;
            }
        }
        mine += total[q];
    }
    // exclusive sum over the threads (digits in order)
    s_scan[tid] = mine;
    __syncthreads();
    for (uint32_t o = 1; o < kBlock; o <<= 1) {
        const uint32_t add = tid >= o ? s_scan[tid - o] : 0;
        __syncthreads();
        s_scan[tid] += add;
        __syncthreads();
    }
    uint32_t base = s_scan[tid] - mine;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const uint32_t d = tid * Q + q;
        uint32_t at = base + before[q];
        if (d < digits) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = s_at[w][d];
                s_at[w][d] = at;
                at += c;
            }
        }
        base += total[q];
    }
    __syncthreads();
    // a wavefront's counters are read and advanced by its own lanes only
    for (uint64_t m = w0; m < w1; m += kWave) {
        const uint64_t n = m + lane;
        const bool have = n < w1;
        const uint32_t key = have ? src.key((uint32_t)n) : 0;
        const uint32_t pos = have ? src.pos((uint32_t)n) : 0;
        const uint32_t d = (key >> p.shift) & (digits - 1);
        unsigned long long same = __ballot(have);
        for (int b = 0; b < p.bits; ++b) {
            const unsigned long long one = __ballot((d >> b) & 1u);
            same &= (d >> b) & 1u ? one : ~one;
        }
        const unsigned long long below = same & ((1ull << lane) - 1);
        uint32_t at = 0;
        if (have) at = s_at[wave][d] + (uint32_t)__popcll(below);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (have && below == 0) s_at[wave][d] += (uint32_t)__popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (have) {
            keys[at] = key;
            poss[at] = pos;
        }
    }
}

// first[v] = sorted place of the first token of row v or later, v = 0 .. V.
__global__ __launch_bounds__(kBlock) void row_first_kernel(const uint32_t* keys, uint32_t N, int64_t V,
                                                           uint32_t* first) {
    const int64_t v = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (v > V) return;
    uint32_t lo = 0, hi = N;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < (uint32_t)v) lo = mid + 1;
        else hi = mid;
    }
    first[v] = lo;
}

// One wavefront to 64 vectors of a row.
template <int DT, int GDT, bool ALIGNED>
__global__ __launch_bounds__(kBlock) void embed_bwd_kernel(const void* g, float scale, const uint32_t* first,
                                                           const uint32_t* poss, void* grad, bool add,
                                                           int64_t rows, int64_t D) {
    constexpr int V = Elem<DT>::V;
    const int64_t v = (int64_t)blockIdx.x * kWaves + uniform((int)(threadIdx.x / kWave));
    if (v >= rows) return;
    const uint32_t p0 = first[v], p1 = first[v + 1];
    if (add && p0 == p1) return;
    for (int64_t d0 = (int64_t)(threadIdx.x % kWave) * V; d0 < D; d0 += kWave * V) {
        const int nvalid = (int)((D - d0) < V ? (D - d0) : V);
        float sum[V];
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0.0f;
        for (uint32_t p = p0; p < p1; ++p) {
            const RowVec<DT> r = load_row<DT, ALIGNED>(g, (size_t)poss[p] * (size_t)D + (size_t)d0, nvalid, 0.0f);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += r.get(j);
        }
        const size_t o0 = (size_t)v * (size_t)D + (size_t)d0;
        if constexpr (GDT == DT) {
            RowOut<DT> o;
            RowVec<DT> old = RowVec<DT>::splat(0.0f);
            if (add) old = load_row<DT, ALIGNED>(grad, o0, nvalid, 0.0f);
#pragma unroll
            for (int j = 0; j < V; ++j) o.v[j] = fmaf(scale, sum[j], old.get(j));
            store_row<DT, ALIGNED>(grad, o0, nvalid, o);
        } else {  // bf16 gradients into an fp32 table
            float* out = reinterpret_cast<float*>(grad) + o0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < nvalid) out[j] = fmaf(scale, sum[j], add ? out[j] : 0.0f);
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct SortPlan {
    int passes, bits;
    uint32_t tile, blocks;
};

SortPlan sort_plan(const EmbedShape& s) {
    SortPlan p;
    int kb = 1;
    while (((int64_t)1 << kb) <= s.V) ++kb;  // keys 0 .. V
    p.passes = (kb + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = (kb + p.passes - 1) / p.passes;
    int64_t tile = (s.N + kMaxSortBlocks - 1) / kMaxSortBlocks;
    tile = (tile + kSortTile - 1) / kSortTile * kSortTile;
    p.tile = (uint32_t)tile;
    p.blocks = (uint32_t)((s.N + tile - 1) / tile);
    return p;
}

struct EmbedWs {
    uint32_t *keys[2], *poss[2], *counts, *first;
};

size_t ws_layout(const EmbedShape& s, void* base, EmbedWs* w) {
    const SortPlan p = sort_plan(s);
    char* c = static_cast<char*>(base);
    size_t at = 0;
    const auto take = [&](size_t words) {
        uint32_t* q = reinterpret_cast<uint32_t*>(c + at);
        at += up256(words * 4);
        return q;
    };
    for (int i = 0; i < 2; ++i) {
        w->keys[i] = take((size_t)s.N);
        w->poss[i] = take((size_t)s.N);
    }
    w->counts = take((size_t)p.blocks << p.bits);
    w->first = take((size_t)s.V + 1);
    return at;
}

template <class Src>
hipError_t sort_pass(Src src, const SortPass& p, uint32_t* counts, uint32_t* keys, uint32_t* poss,
                     hipStream_t st) {
    hipLaunchKernelGGL((sort_count_kernel<Src>), dim3(p.blocks), dim3(kBlock), 0, st, src, p, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((sort_scatter_kernel<Src>), dim3(p.blocks), dim3(kBlock), 0, st, src, p, counts, keys,
                       poss);
    return hipGetLastError();
}

template <int DT, int IB>
hipError_t embed_fwd_t(const EmbedShape& s, const void* ids, const void* w, float scale, void* out,
                       hipStream_t st) {
    const Shape c{s.N, 1, s.D, s.dtype};
    const void* ptrs[2] = {w, out};
    const uint32_t vpr = (uint32_t)((s.D + Elem<DT>::V - 1) / Elem<DT>::V);
    const dim3 grid((unsigned)((s.N + kWaves - 1) / kWaves), (vpr + kWave - 1) / kWave);
    if (rows_aligned(c, ptrs, 2))
        hipLaunchKernelGGL((embed_fwd_kernel<DT, IB, true>), grid, dim3(kBlock), 0, st, ids, w, scale, out, s.N,
                           s.V, s.D, vpr);
    else
        hipLaunchKernelGGL((embed_fwd_kernel<DT, IB, false>), grid, dim3(kBlock), 0, st, ids, w, scale, out, s.N,
                           s.V, s.D, vpr);
    return hipGetLastError();
}

template <int DT, int GDT>
hipError_t embed_rows_t(const EmbedShape& s, const void* g, float scale, const EmbedWs& w, const uint32_t* poss,
                        void* grad, bool add, hipStream_t st) {
    const Shape c{s.N, 1, s.D, s.dtype};
    const void* ptrs[2] = {g, grad};
    const dim3 grid((unsigned)((s.V + kWaves - 1) / kWaves));
    if (rows_aligned(c, ptrs, 2))
        hipLaunchKernelGGL((embed_bwd_kernel<DT, GDT, true>), grid, dim3(kBlock), 0, st, g, scale, w.first, poss,
                           grad, add, s.V, s.D);
    else
        hipLaunchKernelGGL((embed_bwd_kernel<DT, GDT, false>), grid, dim3(kBlock), 0, st, g, scale, w.first, poss,
                           grad, add, s.V, s.D);
    return hipGetLastError();
}

}  // namespace

bool embed_fits(const EmbedShape& s) {
    // 32-bit positions, keys and grid sizes; D in vectors along the grid's second dimension
    return s.N < ((int64_t)1 << 31) && s.V < ((int64_t)1 << 31) - 1 && s.D <= ((int64_t)1 << 22) &&
           (s.V + kWaves) / kWaves < ((int64_t)1 << 32) / kBlock && (s.N + kWaves) / kWaves < ((int64_t)1 << 32) / kBlock;
}

hipError_t launch_embed_fwd(const EmbedShape& s, const void* ids, const void* w, float scale, void* out,
                            hipStream_t st) {
    if (s.dtype == DT_F32)
        return s.id_bytes == 8 ? embed_fwd_t<DT_F32, 8>(s, ids, w, scale, out, st)
                               : embed_fwd_t<DT_F32, 4>(s, ids, w, scale, out, st);
    return s.id_bytes == 8 ? embed_fwd_t<DT_BF16, 8>(s, ids, w, scale, out, st)
                           : embed_fwd_t<DT_BF16, 4>(s, ids, w, scale, out, st);
}

size_t embed_ws_bytes(const EmbedShape& s) {
    EmbedWs w;
    return ws_layout(s, nullptr, &w);
}

hipError_t launch_embed_bwd(const EmbedShape& s, const void* ids, const void* g, float scale, void* grad,
                            int grad_dtype, bool add, void* ws, hipStream_t st) {
    EmbedWs w;
    ws_layout(s, ws, &w);
    const SortPlan plan = sort_plan(s);
    SortPass p{(uint32_t)s.N, plan.tile, plan.blocks, 0, plan.bits};
    hipError_t e = s.id_bytes == 8
                       ? sort_pass(KeysFromIds<8>{ids, s.V}, p, w.counts, w.keys[0], w.poss[0], st)
                       : sort_pass(KeysFromIds<4>{ids, s.V}, p, w.counts, w.keys[0], w.poss[0], st);
    int at = 0;
    for (int i = 1; i < plan.passes && e == hipSuccess; ++i, at ^= 1) {
        p.shift = i * plan.bits;
        e = sort_pass(KeysFromPass{w.keys[at], w.poss[at]}, p, w.counts, w.keys[at ^ 1], w.poss[at ^ 1], st);
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(row_first_kernel, dim3((unsigned)((s.V + 1 + kBlock - 1) / kBlock)), dim3(kBlock), 0, st,
                       w.keys[at], (uint32_t)s.N, s.V, w.first);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (s.dtype == DT_F32) return embed_rows_t<DT_F32, DT_F32>(s, g, scale, w, w.poss[at], grad, add, st);
    if (grad_dtype == DT_F32) return embed_rows_t<DT_BF16, DT_F32>(s, g, scale, w, w.poss[at], grad, add, st);
    return embed_rows_t<DT_BF16, DT_BF16>(s, g, scale, w, w.poss[at], grad, add, st);
}

}  // namespace lrscan
