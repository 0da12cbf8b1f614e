// gated_fused.hip -- the gated scan in one launch, in tiles, with a look-back
// (the form of fused.hip; tickets, workspace and waiting in fused_common.hpp).
//
// Forward: a thread loads its rows of x and of both gates, forms (a, b) of
// every step once (gated_math.hpp) and keeps them in registers from the
// summary of its rows to the replay, so no gate is evaluated twice.
//
// Reverse: the summary needs a and grad_out only.  The replay recomputes the
// gates from the rows kept in storage form (an fp32 copy of every coefficient
// would not fit beside them) and writes the three gradients; the tile's sum
// of P for the decay gradient goes to one partial row for each tile.
//
// Bound (MI355X, bf16 [8, 2048, 2560] with resets, caches flushed): forward
// 74 us for 336 MB (4.5 TB/s; a copy reaches 4.95), with the vector units busy
// for 46 of them, 37 instructions an element of which 6 are transcendental;
// reverse 152 us for 671 MB (4.4 TB/s), 78 of them busy, 64 instructions an
// element.  fp32, with half the elements to a byte, runs at the memory's rate:
// reverse [4, 2048, 4096] 195 us for 1.07 GB (5.5 TB/s).
//
// A reset step is a map that drops its argument.  It is carried as the map
// (p, q) with p = -0: a product of transitions is never -0, because each
// is >= +0 and a reset enters compositions by selects, so the sign tells a
// drop from a product that underflowed, whose argument still counts where it
// is an infinity or NaN.
#include <type_traits>

#include "fused_common.hpp"
#include "gated.hpp"
#include "gated_geo.hpp"
#include "gated_math.hpp"

namespace lrscan {

namespace {

constexpr uint32_t kDropBits = 0x80000000u;  // -0.0f
__device__ __forceinline__ bool drops(Aff m) { return __float_as_uint(m.p) == kDropBits; }

// Composition and application of maps, with resets (RST) or without.
template <bool RST>
struct GatedThen {
    __device__ __forceinline__ static Aff then(Aff e, Aff l) {
        const Aff m = aff_then(e, l);
        if constexpr (RST) return drops(l) ? l : m;
        return m;
    }
};
template <bool RST>
__device__ __forceinline__ float gated_apply(Aff m, float h) {
    const float x = aff_apply(m, h);
    if constexpr (RST) return drops(m) ? m.q : x;
    return x;
}

__device__ __forceinline__ unsigned long long pack_map(Aff m) {
    return (unsigned long long)publishable(m.p) | ((unsigned long long)publishable(m.q) << 32);
}
__device__ __forceinline__ Aff unpack_map(unsigned long long w) {
    return Aff{__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

// A published entry: (P, Q) in one 64-bit word, H in one 32-bit word.
template <bool RST>
struct GatedLink {
    using S = float;
    using M = Aff;
    using HRaw = uint32_t;
    using MRaw = unsigned long long;
    const uint32_t* hs;
    const unsigned long long* pqs;
    int nS, s, W, c;
    __device__ size_t entry(int j) const { return ((size_t)j * (size_t)nS + (size_t)s) * W + c; }
    __device__ HRaw load_h(int j) const { return peek_u32(hs + entry(j)); }
    __device__ MRaw load_m(int j) const { return peek_u64(pqs + entry(j)); }
    __device__ static HRaw empty_h() { return kEmpty; }
    __device__ static MRaw empty_m() { return ~0ull; }
    __device__ static bool ready_h(HRaw w) { return w != kEmpty; }
    __device__ static bool ready_m(MRaw w) { return (uint32_t)w != kEmpty; }
    __device__ static S state(HRaw w) { return __uint_as_float(w); }
    __device__ static M map(MRaw w) { return unpack_map(w); }
    __device__ static S apply(M m, S x) { return gated_apply<RST>(m, x); }
};
constexpr int kGatedWords = 3;  // (P, Q) and H

struct GatedFwdArgs {
    GatedFwd p;
    Scratch sc;
    Dims d;
    uint32_t polls;
};
struct GatedBwdArgs {
    GatedBwd p;
    float* part;  // [NK * B, D] sums of P over a tile's rows, or NULL
    Scratch sc;
    Dims d;
    uint32_t polls;
};

template <class C, int RK>
__device__ __forceinline__ RowVec<C::DT> load_tile(const char* base, uint32_t off, int nvalid) {
    if constexpr (RK == kWhole) {
        RowVec<C::DT> r;
        r.w = load16_any(base + off);
        return r;
    } else {
        return load_vec<C::DT, RK == kAligned, true>(base, off, nvalid, 0.0f);
    }
}
template <class C, int RK>
__device__ __forceinline__ void store_tile(char* base, uint32_t off, int nvalid, const RowOut<C::DT>& o) {
    if constexpr (RK == kWhole) store16_any(base + off, o.pack());
    else store_vec<C::DT, RK == kAligned>(base, off, nvalid, o);
}

// Whether every row of the tile and some column of every vector exist.
template <class C>
__device__ __forceinline__ bool tile_full(const Geo& g, const Dims& d) {
    return g.trow0 + C::CT <= d.T && g.dcol0 + (C::TPR - 1) * C::V < d.D;
}

// One operand's rows of a tile: base of (batch row, first row, first lane) and
// the bytes between rows, 32-bit inside a tile.
struct TileRows {
    char* p;
    uint32_t st;
    template <class C, int RK>
    __device__ __forceinline__ static TileRows of(const Rows& r, const Geo& g) {
        return TileRows{r.row(g.bi, g.trow0) + (size_t)g.dcol0 * C::EB - (RK == kWhole ? 16 : 0), (uint32_t)r.st};
    }
    __device__ __forceinline__ uint32_t off(const Geo& g, int row, int T) const {
        return row_off(g, row, T, st);
    }
};

// The map of step t of one lane, forward and reverse, and its place in a fold.
template <bool RST>
__device__ __forceinline__ void fold_fwd(Aff& m, GatedStep s, bool start) {
    const Aff n{s.a * m.p, fmaf(s.a, m.q, s.b)};
    m = RST && start ? Aff{-0.0f, s.b} : n;
}
template <bool RST>
__device__ __forceinline__ void fold_rev(Aff& m, float a, float g, bool start) {
    const Aff n{a * m.p, a * (m.q + g)};
    m = RST && start ? Aff{-0.0f, 0.0f} : n;
}
template <bool RST>
__device__ __forceinline__ GatedStep gated_coef(float x, float gr, float gi, float rate, bool start) {
    const GatedStep s = gated_step_of(x, gr, gi, rate);
    if constexpr (RST) {
        if (start) return gated_start_of(x, gi);
    }
    return s;
}

// Map of tile j of series (bi, lane block) for lane `col`, in exactly the
// order the workgroup that owns tile j computes it.
template <class C, bool RST>
__device__ Aff gated_fwd_tile_map(const GatedFwdArgs& x, int j, int bi, int col) {
    constexpr int NR = C::NR, RG = C::RG, SEGS = C::WAVES * C::RG;
    Aff A = aff_identity(), Wv = aff_identity();
    if (col >= x.d.D) return A;
    const float rate = gate_rate(x.p.decay[col], x.p.scale);
#pragma unroll 1
    for (int sg = 0; sg < SEGS; ++sg) {
        Aff t = aff_identity();
        const int r0 = j * C::CT + sg * NR;
#pragma unroll 1
        for (int i = 0; i < NR; ++i) {
            const int r = r0 + i;
            if (r < x.d.T) {
                const bool start = RST && x.p.reset[(size_t)bi * x.d.T + r];
                const GatedStep s = gated_coef<RST>(Elem<C::DT>::load1(x.p.x.row(bi, r), col),
                                                    Elem<C::DT>::load1(x.p.gr.row(bi, r), col),
                                                    Elem<C::DT>::load1(x.p.gi.row(bi, r), col), rate, start);
                fold_fwd<RST>(t, s, start);
            } else {
                fold_fwd<RST>(t, GatedStep{1.0f, 0.0f}, false);
            }
        }
        Wv = GatedThen<RST>::then(Wv, t);
        if (sg % RG == RG - 1) {  // a wavefront's segments, then the wavefronts in order
            A = GatedThen<RST>::then(A, Wv);
            Wv = aff_identity();
        }
    }
    return unpack_map(pack_map(A));
}

template <class C, bool RST, bool LAST>
__device__ Aff gated_bwd_tile_map(const GatedBwdArgs& x, int j, int bi, int col) {
    constexpr int NR = C::NR, RG = C::RG, SEGS = C::WAVES * C::RG;
    Aff A = aff_identity(), Wv = aff_identity();
    if (col >= x.d.D) return A;
    const float rate = gate_rate(x.p.decay[col], x.p.scale);
#pragma unroll 1
    for (int sg = SEGS - 1; sg >= 0; --sg) {
        Aff t = aff_identity();
        const int r0 = j * C::CT + sg * NR;
        if (LAST && r0 < x.d.T && r0 + NR >= x.d.T) t.q = x.p.grad_last[(size_t)bi * x.d.D + col];
#pragma unroll 1
        for (int i = NR - 1; i >= 0; --i) {
            const int r = r0 + i;
            if (r < x.d.T) {
                const bool start = RST && x.p.reset && x.p.reset[(size_t)bi * x.d.T + r];
                const float a = gated_a_of(Elem<C::DT>::load1(x.p.gr.row(bi, r), col), rate);
                const float g = Elem<C::DT>::load1(x.p.g, ((size_t)bi * x.d.T + r) * (size_t)x.d.D + col);
                fold_rev<RST>(t, a, g, start);
            } else {
                fold_rev<RST>(t, 1.0f, 0.0f, false);
            }
        }
        Wv = GatedThen<RST>::then(Wv, t);
        if (sg % RG == 0) {  // a wavefront's segments (last first), then the wavefronts
            A = GatedThen<RST>::then(A, Wv);
            Wv = aff_identity();
        }
    }
    return unpack_map(pack_map(A));
}

// Rates of the tile's lanes (lanes past D take the last one's; never used).
template <class C, int RK>
__device__ __forceinline__ void tile_rates(float (&s_rate)[C::W], const float* decay, float scale,
                                           const Geo& g, int D) {
    if (threadIdx.x < C::W) {
        const int c = slot_column<C, RK>(g, (int)threadIdx.x, D);
        s_rate[threadIdx.x] = gate_rate(decay[c < D ? c : D - 1], scale);
    }
    __syncthreads();
}

// Segment starts among this thread's rows that exist, bit i for row i.
template <class C>
__device__ __forceinline__ uint32_t start_bits(const uint8_t* reset, const Geo& g, int T) {
    static_assert(C::NR % 4 == 0 || C::NR < 4, "whole words of mask bytes");
    uint32_t bits = 0;
    if (C::NR % 4 == 0 && g.nrows == C::NR) {
        const uint8_t* p = reset + (size_t)g.bi * T + g.row0;
#pragma unroll
        for (int w = 0; w < C::NR / 4; ++w) {
            uint32_t four;
            __builtin_memcpy(&four, p + 4 * w, 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) bits |= ((four >> (8 * i)) & 0xffu ? 1u : 0u) << (4 * w + i);
        }
        return bits;
    }
#pragma unroll
    for (int i = 0; i < C::NR; ++i)
        if (i < g.nrows && reset_byte(reset, g, i, T)) bits |= 1u << i;
    return bits;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// OUT = false: state-only forward: only the thread holding row T-1 replays.
template <class C, int RK, bool RST, bool OUT>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::OCC_F)))
void gated_fwd_kernel(GatedFwdArgs x) {
    constexpr int V = C::V, W = C::W, RG = C::RG, NR = C::NR, TPR = C::TPR;
    constexpr int SEGS = C::WAVES * RG;
    using Link = GatedLink<RST>;
    __shared__ Aff s_seg[SEGS][W];  // each segment's map, then its wavefront's maps before it composed
    __shared__ Aff s_wav[C::WAVES][W];  // each wavefront's map, then the wavefronts' before it composed
    __shared__ float s_hin[W];      // the state entering the tile, per lane
    __shared__ float s_rate[W];

    const Dims d = x.d;
    const int tid = threadIdx.x;
    const int wave = uniform((int)(threadIdx.x / kWave));
    const int l = tid % kWave;
    const int rg = l / TPR;
    const int cg = l % TPR;
    const Ticket tk = take_ticket(x.sc);
    const Geo g = gated_geo<C, RK, false>(tk.ticket, d, wave, rg, cg);
    const TileRows px = TileRows::of<C, RK>(x.p.x, g), pr = TileRows::of<C, RK>(x.p.gr, g),
                   pi = TileRows::of<C, RK>(x.p.gi, g);
    char* po = static_cast<char*>(x.p.out) + g.tbase;
    const uint32_t rowbytes = (uint32_t)d.D * C::EB;

    const uint32_t rbits = RST ? start_bits<C>(x.p.reset, g, d.T) : 0u;
    RowVec<C::DT> rx[NR], rr[NR], ri[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = g.row0 + i;
        rr[i] = load_tile<C, RK>(pr.p, pr.off(g, row, d.T), g.nvalid);
        ri[i] = load_tile<C, RK>(pi.p, pi.off(g, row, d.T), g.nvalid);
        rx[i] = load_tile<C, RK>(px.p, px.off(g, row, d.T), g.nvalid);
    }
    tile_rates<C, RK>(s_rate, x.p.decay, x.p.scale, g, d.D);
    float rate[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rate[j] = s_rate[cg * V + j];

    // Coefficients and summary, row by row.  Segment starts and rows that do not
    // exist are put right under wavefront-wide branches, as few rows have them,
    // rather than by selects for every element ([8, 2048, 2560] bf16 with a start
    // every 512 tokens: 85 -> 74 us; folding such a wavefront's rows twice: 76).
    const bool full = tile_full<C>(g, d);
    float ca[NR][V], cb[NR][V];
    Aff m[V];
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = aff_identity();
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const bool start = RST && ((rbits >> i) & 1u), gone = i >= g.nrows;
        const bool starts = RST && __any(start);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const GatedStep s = gated_step_of(rx[i].get(j), rr[i].get(j), ri[i].get(j), rate[j]);
            ca[i][j] = s.a;
            cb[i][j] = s.b;
        }
        if (starts) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const GatedStep s = gated_start_of(rx[i].get(j), ri[i].get(j));
                ca[i][j] = start ? s.a : ca[i][j];
                cb[i][j] = start ? s.b : cb[i][j];
            }
        }
        if (!full) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                ca[i][j] = gone ? 1.0f : ca[i][j];
                cb[i][j] = gone ? 0.0f : cb[i][j];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            m[j].p = ca[i][j] * m[j].p;
            m[j].q = fmaf(ca[i][j], m[j].q, cb[i][j]);
        }
        if (starts) {
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] = start ? Aff{-0.0f, cb[i][j]} : m[j];
        }
    }
    const int seg = wave * RG + rg;
#pragma unroll
    for (int j = 0; j < V; ++j) s_seg[seg][cg * V + j] = m[j];
    fold_wave_segments<C, false, GatedThen<RST>>(s_seg, s_wav, wave, l, aff_identity());
    const uint32_t phase = tk.phase;
    const unsigned long long* pqs = reinterpret_cast<const unsigned long long*>(x.sc.region[phase]);
    const uint32_t* hs = x.sc.region[phase] + 2 * x.sc.entries;
    EarlyWindow<Link, C::EW> early;
    if (tid < W) {
        int z = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) z += zero_after(m[j].q);
        early.template take<-1>(Link{hs, pqs, d.nS, g.s, W, tid + z}, g.k, d.NK);
    }
    __syncthreads();

    // exclusive prefixes and tile map, publication, look-back: one lane per thread
    if (tid < W) {
        const int c = tid;
        Aff A = aff_identity();
#pragma unroll
        for (int w = 0; w < C::WAVES; ++w) {
            const Aff t = s_wav[w][c];
            s_wav[w][c] = A;
            A = GatedThen<RST>::then(A, t);
        }
        const size_t o = ((size_t)g.k * (size_t)d.nS + (size_t)g.s) * W + c;
        const bool more = g.k + 1 < d.NK;
        if (more) publish_u64(const_cast<unsigned long long*>(pqs) + o, pack_map(A));
        const int dl = slot_column<C, RK>(g, c, d.D);
        const float base0 = (x.p.h0 && dl < d.D) ? x.p.h0[(size_t)g.bi * d.D + dl] : 0.0f;
        const Link lk{hs, pqs, d.nS, g.s, W, c};
        float hin;
        if (!early.template resolve<-1>(g.k, d.NK, base0, &hin))
            hin = look_back<Link, -1, C::LB>(lk, g.k, d.NK, base0, x.polls, [&](int j) {
                return gated_fwd_tile_map<C, RST>(x, j, g.bi, dl);
            });
        if (more) publish_u32(const_cast<uint32_t*>(hs) + o, publishable(gated_apply<RST>(A, hin)));
        s_hin[c] = hin;
    }
    __syncthreads();
    clear_share(x.sc, tk.phase, tk.nclear, C::NT, tk.ticket);

    const bool ends = g.nrows > 0 && g.row0 + g.nrows == d.T;  // holds row T-1
    if constexpr (!OUT) {
        if (!(x.p.last && ends)) return;
    }
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        h[j] = gated_apply<RST>(s_seg[seg][cg * V + j],
                                gated_apply<RST>(s_wav[wave][cg * V + j], s_hin[cg * V + j]));
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const bool start = RST && ((rbits >> i) & 1u);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float n = fmaf(ca[i][j], h[j], cb[i][j]);  // (of a row that does not exist: h itself)
            h[j] = n;
        }
        if (RST && __any(start)) {
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = start ? cb[i][j] : h[j];
        }
        if (OUT && (full || i < g.nrows)) {
            RowOut<C::DT> o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.v[j] = h[j];
            store_tile<C, RK>(po, row_off(g, g.row0 + i, d.T, rowbytes), g.nvalid, o);
        }
    }
    if (x.p.last && ends) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < g.nvalid) x.p.last[(size_t)g.bi * d.D + g.d0 + j] = h[j];
    }
}

// ---------------------------------------------------------------------------
// reverse time
// ---------------------------------------------------------------------------
// LAST: the last state has a gradient (RST, whose resets may be absent then).
// It is added to the last row's gradient and does not enter as a carry: as a
// carry it would be multiplied on its own, and where it cancels that row's
// gradient the sum would keep the products' roundings.  (In one version with
// the rest: 153 against 148 us at bf16 [8,2048,2560].)
template <class C, int RK, bool RST, bool LAST>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::OCC_G)))
void gated_bwd_kernel(GatedBwdArgs x) {
    constexpr int V = C::V, W = C::W, RG = C::RG, NR = C::NR, TPR = C::TPR;
    constexpr int SEGS = C::WAVES * RG;
    using Link = GatedLink<RST>;
    __shared__ Aff s_seg[SEGS][W];
    __shared__ Aff s_wav[C::WAVES][W];
    __shared__ float s_cin[W];
    __shared__ float s_rate[W];

    const Dims d = x.d;
    const int tid = threadIdx.x;
    const int wave = uniform((int)(threadIdx.x / kWave));
    const int l = tid % kWave;
    const int rg = l / TPR;
    const int cg = l % TPR;
    const Ticket tk = take_ticket(x.sc);
    const Geo g = gated_geo<C, RK, true>(tk.ticket, d, wave, rg, cg);
    const uint32_t rowbytes = (uint32_t)d.D * C::EB;
    const TileRows px = TileRows::of<C, RK>(x.p.x, g), pr = TileRows::of<C, RK>(x.p.gr, g),
                   pi = TileRows::of<C, RK>(x.p.gi, g);
    const TileRows qx = TileRows::of<C, RK>(x.p.gx, g), qr = TileRows::of<C, RK>(x.p.ggr, g),
                   qi = TileRows::of<C, RK>(x.p.ggi, g);
    const char* pg = static_cast<const char*>(x.p.g) + g.tbase;
    const int hrow0 = g.trow0 > 0 ? g.trow0 - 1 : 0;  // h_{t-1} is row t-1 of `out`
    const char* ph = static_cast<const char*>(x.p.out) + g.tbase - (size_t)(g.trow0 - hrow0) * rowbytes;

    const uint32_t rbits = RST && (!LAST || x.p.reset) ? start_bits<C>(x.p.reset, g, d.T) : 0u;
    // what the summary uses first, in its order, then the replay's rows
    RowVec<C::DT> rr[NR], rg_[NR], rx[NR], ri[NR], rh[NR];
#pragma unroll
    for (int i = NR - 1; i >= 0; --i) {
        const int row = g.row0 + i;
        rr[i] = load_tile<C, RK>(pr.p, pr.off(g, row, d.T), g.nvalid);
        rg_[i] = load_tile<C, RK>(pg, row_off(g, row, d.T, rowbytes), g.nvalid);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = NR - 1; i >= 0; --i) {
        const int row = g.row0 + i;
        const int rc = row < d.T ? row : d.T - 1;
        const int hr = rc >= 1 ? rc - 1 : 0;
        rh[i] = load_tile<C, RK>(ph, (uint32_t)(hr - hrow0) * rowbytes + g.coff, g.nvalid);
        rx[i] = load_tile<C, RK>(px.p, px.off(g, row, d.T), g.nvalid);
        ri[i] = load_tile<C, RK>(pi.p, pi.off(g, row, d.T), g.nvalid);
    }
    __builtin_amdgcn_sched_barrier(0);
    tile_rates<C, RK>(s_rate, x.p.decay, x.p.scale, g, d.D);
    float rate[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rate[j] = s_rate[cg * V + j];

    // reverse summary: the map from the carry entering the segment on the
    // right to the carry a_s lambda_s leaving its first row s
    const bool full = tile_full<C>(g, d) && !(LAST && g.k == d.NK - 1);
    const auto entering = [&](int j) {
        if constexpr (LAST) {
            if (g.nrows > 0 && g.row0 + g.nrows == d.T && j < g.nvalid)
                return x.p.grad_last[(size_t)g.bi * d.D + g.d0 + j];
        }
        return 0.0f;
    };
    Aff m[V];
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = aff_identity();
#pragma unroll
    for (int i = NR - 1; i >= 0; --i) {
        const bool start = RST && ((rbits >> i) & 1u);
#pragma unroll
        for (int j = 0; j < V; ++j)
            fold_rev<false>(m[j], gated_a_of(rr[i].get(j), rate[j]), rg_[i].get(j), false);
        if (RST && __any(start)) {
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] = start ? Aff{-0.0f, 0.0f} : m[j];
        }
    }
    if (!full) {  // folded again, without the rows that do not exist
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = Aff{1.0f, entering(j)};
#pragma unroll
        for (int i = NR - 1; i >= 0; --i) {
            opaque(rr[i]);
            opaque(rg_[i]);
            const bool start = RST && ((rbits >> i) & 1u), gone = i >= g.nrows;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float a = gated_a_of(rr[i].get(j), rate[j]), gt = rg_[i].get(j);
                fold_rev<RST>(m[j], gone ? 1.0f : a, gone ? 0.0f : gt, start);
            }
        }
    }
    const int seg = wave * RG + rg;
#pragma unroll
    for (int j = 0; j < V; ++j) s_seg[seg][cg * V + j] = m[j];
    fold_wave_segments<C, true, GatedThen<RST>>(s_seg, s_wav, wave, l, aff_identity());
    const uint32_t phase = tk.phase;
    const unsigned long long* pqs = reinterpret_cast<const unsigned long long*>(x.sc.region[phase]);
    const uint32_t* hs = x.sc.region[phase] + 2 * x.sc.entries;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        opaque(rr[i]);
        opaque(rg_[i]);
    }
    EarlyWindow<Link, C::EW> early;
    if (tid < W) {
        int z = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) z += zero_after(m[j].q);
        early.template take<+1>(Link{hs, pqs, d.nS, g.s, W, tid + z}, g.k, d.NK);
    }
    __syncthreads();

    if (tid < W) {
        const int c = tid;
        Aff A = aff_identity();
#pragma unroll
        for (int w = C::WAVES - 1; w >= 0; --w) {
            const Aff t = s_wav[w][c];
            s_wav[w][c] = A;
            A = GatedThen<RST>::then(A, t);
        }
        const size_t o = ((size_t)g.k * (size_t)d.nS + (size_t)g.s) * W + c;
        const bool more = g.k > 0;
        if (more) publish_u64(const_cast<unsigned long long*>(pqs) + o, pack_map(A));
        const int dl = slot_column<C, RK>(g, c, d.D);
        const Link lk{hs, pqs, d.nS, g.s, W, c};
        float cin;
        if (!early.template resolve<+1>(g.k, d.NK, 0.0f, &cin))
            cin = look_back<Link, +1, C::LB>(lk, g.k, d.NK, 0.0f, x.polls, [&](int j) {
                return gated_bwd_tile_map<C, RST, LAST>(x, j, g.bi, dl);
            });
        if (more) publish_u32(const_cast<uint32_t*>(hs) + o, publishable(gated_apply<RST>(A, cin)));
        s_cin[c] = cin;
    }
    __syncthreads();
    clear_share(x.sc, tk.phase, tk.nclear, C::NT, tk.ticket);

    float carry[V], sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        carry[j] = gated_apply<RST>(s_seg[seg][cg * V + j],
                                    gated_apply<RST>(s_wav[wave][cg * V + j], s_cin[cg * V + j]));
        sum[j] = 0.0f;
    }
    if (LAST && !full) {
#pragma unroll
        for (int j = 0; j < V; ++j) carry[j] += entering(j);
    }
    // One row; STARTS: some thread of the wavefront has a segment start there (as
    // a version of its own: the selects under a branch in one version spilled,
    // 166 against 158 us).
    const auto replay = [&](int i, auto starts) {
        constexpr bool STARTS = decltype(starts)::value;
        const int row = g.row0 + i;
        const bool start = STARTS && ((rbits >> i) & 1u);
        RowOut<C::DT> ox, orr, oi;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float lam = carry[j] + rg_[i].get(j);
            float hp = rh[i].get(j);
            if (i == 0 && g.row0 == 0)  // row 0: h0, or 0
                hp = (x.p.h0 && j < g.nvalid) ? x.p.h0[(size_t)g.bi * d.D + g.d0 + j] : 0.0f;
            const float xv = rx[i].get(j), iv = ri[i].get(j), rv = rr[i].get(j);
            GatedGrad q = gated_grad_of(xv, rv, iv, rate[j], hp, lam);
            carry[j] = q.a * lam;
            if (start) {
                q = gated_start_grad_of(xv, iv, lam);
                carry[j] = 0.0f;
            }
            ox.v[j] = q.dx;
            orr.v[j] = q.dgr;
            oi.v[j] = q.dgi;
            sum[j] += q.p;
        }
        store_tile<C, RK>(qx.p, qx.off(g, row, d.T), g.nvalid, ox);
        store_tile<C, RK>(qr.p, qr.off(g, row, d.T), g.nvalid, orr);
        store_tile<C, RK>(qi.p, qi.off(g, row, d.T), g.nvalid, oi);
    };
#pragma unroll
    for (int i = NR - 1; i >= 0; --i) {
        if (full || i < g.nrows) {
            if (RST && __any((rbits >> i) & 1u)) replay(i, std::true_type{});
            else replay(i, std::false_type{});
        }
    }
    if (x.p.grad_h0 && g.nrows > 0 && g.row0 == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < g.nvalid) x.p.grad_h0[(size_t)g.bi * d.D + g.d0 + j] = carry[j];
    }
    if (!x.part) return;
    // the tile's sum of P for each lane: a wavefront's segments in order, then
    // the wavefronts (s_seg and s_wav have been read; a wavefront reads back
    // only its own rows of s_seg)
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) s_seg[seg][cg * V + j].p = sum[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int q = 0; q < (W + kWave - 1) / kWave; ++q) {
        const int c = q * kWave + l;
        if (W < kWave && c >= W) break;
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < RG; ++r) t += s_seg[wave * RG + r][c].p;
        s_wav[wave][c].p = t;
    }
    __syncthreads();
    const int dt = tid < W ? slot_column<C, RK>(g, tid, d.D) : d.D;
    if (dt < d.D) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < C::WAVES; ++w) t += s_wav[w][tid].p;
        const int nB = d.nS / d.nW;
        x.part[((size_t)g.k * nB + g.bi) * (size_t)d.D + dt] = t;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// OCC_F, OCC_G: wavefronts a SIMD is to hold, forward and reverse (their
// registers fit without spilling, or with at most 56 bytes).
template <int DT, int TPR, int NR, int LB, int OF, int OB>
struct GCfg : Cfg<DT, TPR, NR, 4, LB> {
    static constexpr int OCC_F = OF, OCC_G = OB;
};
template <int DT> using Tile16x32 = GCfg<DT, 16, 2, 4, 5, 4>;
template <int DT> using Tile16x64 = GCfg<DT, 16, 4, 4, 3, 3>;
template <int DT> using Tile8x128 = GCfg<DT, 8, 4, 8, 3, 3>;
template <int DT> using Tile8x256 = GCfg<DT, 8, 8, 8, 2, 2>;

// Tile of a shape: `width` threads of 16 bytes along a row, `tile` rows.
//
// Measured on MI355X (us forward / reverse, caches flushed; 16x32, 16x64,
// 8x128, 8x256):
//   bf16 [512,32,2560]   75/145  104/217  201/370  388/709
//   bf16 [256,64,2560]   77/154   68/142  112/211  203/367
//   bf16 [64,200,2560]   67/130   66/134   68/134   70/127
//   bf16 [8,2048,2560]     -      74/153   75/151   77/151
//   bf16 [1,131072,1024]   -     572/ -   251/ -   236/ -
//   bf16 [1,131072,256]    -      - /503    - /212   - /152
//   bf16 [1,4096,2560]   49/62    35/57    30/57    34/61
//   f32  [4,2048,4096]     -      97/214   95/194   93/193
// So a tile is no taller than a short sequence.  Otherwise few chains of tall
// tiles: a chain hands its state on about every 0.28 us, so 64-row tiles want
// some 64 chains of them to keep the memory busy, and tall ones enough tiles
// (2048) to fill the GPU evenly.  With many chains the bf16 forward is fastest
// in wide tiles: its arithmetic is as long as its loads, and 64 rows leave
// registers for a third wavefront to overlap them.
struct GatedTile {
    int width, tile;
};
GatedTile gated_tile(const Shape& s, int dir) {
    const int64_t row = s.D * (s.dtype == DT_F32 ? 4 : 2);
    const int64_t chains16 = s.B * ((row + 255) / 256), chains8 = s.B * ((row + 127) / 128);
    const bool wide = row > 128;
    if (s.D < (s.dtype == DT_F32 ? Elem<DT_F32>::V : Elem<DT_BF16>::V)) return GatedTile{8, 128};  // kNarrow
    if (s.T <= 32 && wide) return GatedTile{16, 32};
    if (s.T <= 64 && wide) return GatedTile{16, 64};
    if (dir == 0 && s.dtype == DT_BF16 && wide && chains16 >= 64) return GatedTile{16, 64};
    const int64_t tall = (s.T + 255) / 256;
    if (chains8 * tall >= 2048 && tall * 256 <= s.T + s.T / 4) return GatedTile{8, 256};
    return GatedTile{8, 128};
}

template <class C, int RK>
void fwd_cfg(const GatedFwdArgs& x, hipStream_t st) {
    const dim3 grid(x.sc.total_tiles), block(C::NT);
    if (x.p.out) {
        if (x.p.reset) hipLaunchKernelGGL((gated_fwd_kernel<C, RK, true, true>), grid, block, 0, st, x);
        else hipLaunchKernelGGL((gated_fwd_kernel<C, RK, false, true>), grid, block, 0, st, x);
    } else {
        if (x.p.reset) hipLaunchKernelGGL((gated_fwd_kernel<C, RK, true, false>), grid, block, 0, st, x);
        else hipLaunchKernelGGL((gated_fwd_kernel<C, RK, false, false>), grid, block, 0, st, x);
    }
}

template <class C, int RK>
void bwd_cfg(const GatedBwdArgs& x, hipStream_t st) {
    const dim3 grid(x.sc.total_tiles), block(C::NT);
    if (x.p.grad_last) hipLaunchKernelGGL((gated_bwd_kernel<C, RK, true, true>), grid, block, 0, st, x);
    else if (x.p.reset) hipLaunchKernelGGL((gated_bwd_kernel<C, RK, true, false>), grid, block, 0, st, x);
    else hipLaunchKernelGGL((gated_bwd_kernel<C, RK, false, false>), grid, block, 0, st, x);
}

template <int DT, int RK>
void fwd_rk(const GatedTile& t, const GatedFwdArgs& x, hipStream_t st) {
    if (t.tile == 32) fwd_cfg<Tile16x32<DT>, RK>(x, st);
    else if (t.tile == 64) fwd_cfg<Tile16x64<DT>, RK>(x, st);
    else if (t.tile == 128) fwd_cfg<Tile8x128<DT>, RK>(x, st);
    else fwd_cfg<Tile8x256<DT>, RK>(x, st);
}
template <int DT, int RK>
void bwd_rk(const GatedTile& t, const GatedBwdArgs& x, hipStream_t st) {
    if (t.tile == 32) bwd_cfg<Tile16x32<DT>, RK>(x, st);
    else if (t.tile == 64) bwd_cfg<Tile16x64<DT>, RK>(x, st);
    else if (t.tile == 128) bwd_cfg<Tile8x128<DT>, RK>(x, st);
    else bwd_cfg<Tile8x256<DT>, RK>(x, st);
}
template <int DT>
void fwd_t(const GatedTile& t, bool al, const GatedFwdArgs& x, hipStream_t st) {
    if (al) fwd_rk<DT, kAligned>(t, x, st);
    else if (x.d.D >= Elem<DT>::V) fwd_rk<DT, kWhole>(t, x, st);
    else fwd_cfg<Tile8x128<DT>, kNarrow>(x, st);
}
template <int DT>
void bwd_t(const GatedTile& t, bool al, const GatedBwdArgs& x, hipStream_t st) {
    if (al) bwd_rk<DT, kAligned>(t, x, st);
    else if (x.d.D >= Elem<DT>::V) bwd_rk<DT, kWhole>(t, x, st);
    else bwd_cfg<Tile8x128<DT>, kNarrow>(x, st);
}

Layout gated_layout(const GatedShape& s, int dir) {
    const Shape c{s.B, s.T, s.D, s.dtype};
    const GatedTile t = gated_tile(c, dir);
    return layout_of(c, t.width, t.tile);
}

// Byte offsets inside a tile, and to its rows, in 32 bits.
bool rows_fit(const GatedShape& s, size_t st, int tile) {
    return s.T == 1 || st * (size_t)(tile + 1) < ((size_t)1 << 31);
}

}  // namespace

bool gated_fused_fits(const GatedShape& s, int dir, const size_t* row_strides, int n) {
    const Shape c{s.B, s.T, s.D, s.dtype};
    const GatedTile t = gated_tile(c, dir);
    const int64_t eb = s.dtype == DT_F32 ? 4 : 2;
    if (!rows_fit(s, (size_t)(s.D * eb), t.tile)) return false;
    for (int i = 0; i < n; ++i)
        if (!rows_fit(s, row_strides[i], t.tile)) return false;
    if (s.T >= ((int64_t)1 << 31) - 2 * t.tile || s.D >= ((int64_t)1 << 29)) return false;
    const Layout L = layout_of(c, t.width, t.tile);
    if (s.B * ((s.D + L.W - 1) / L.W) >= ((int64_t)1 << 31)) return false;
    if ((unsigned long long)((s.T + t.tile - 1) / t.tile) * (unsigned long long)(s.B * ((s.D + L.W - 1) / L.W)) >=
        0xffffffffull)
        return false;
    return grid_fits(L, 4 * kWave);
}

size_t gated_fused_bytes(const GatedShape& s) {
    size_t most = 0;
    for (int dir = 0; dir < 2; ++dir)
        most = std::max(most, kHeaderBytes + 2 * region_bytes_for(gated_layout(s, dir), kGatedWords));
    return most;
}

int64_t gated_fused_part_rows(const GatedShape& s) { return (int64_t)gated_layout(s, 1).NK * s.B; }

hipError_t launch_gated_fused_fwd(const GatedShape& s, const GatedFwd& p, void* ws, size_t ws_bytes,
                                  bool init, int polls, hipStream_t st) {
    const Layout L = gated_layout(s, 0);
    GatedFwdArgs x;
    const hipError_t e = prepare(ws, ws_bytes, init, L, kGatedWords, st, &x.sc);
    if (e != hipSuccess) return e;
    x.p = p;
    x.d = Dims{(int)s.T, (int)s.D, L.nW, L.nS, L.NK};
    x.polls = polls > 0 ? (uint32_t)polls : kDefaultPolls;
    const bool al = gated_fwd_aligned(s, p);
    const GatedTile t = gated_tile(Shape{s.B, s.T, s.D, s.dtype}, 0);
    if (s.dtype == DT_F32) fwd_t<DT_F32>(t, al, x, st);
    else fwd_t<DT_BF16>(t, al, x, st);
    return hipGetLastError();
}

hipError_t launch_gated_fused_bwd(const GatedShape& s, const GatedBwd& p, float* part, void* ws,
                                  size_t ws_bytes, bool init, int polls, hipStream_t st) {
    const Layout L = gated_layout(s, 1);
    GatedBwdArgs x;
    const hipError_t e = prepare(ws, ws_bytes, init, L, kGatedWords, st, &x.sc);
    if (e != hipSuccess) return e;
    x.p = p;
    x.part = part;
    x.d = Dims{(int)s.T, (int)s.D, L.nW, L.nS, L.NK};
    x.polls = polls > 0 ? (uint32_t)polls : kDefaultPolls;
    const bool al = gated_bwd_aligned(s, p);
    const GatedTile t = gated_tile(Shape{s.B, s.T, s.D, s.dtype}, 1);
    if (s.dtype == DT_F32) bwd_t<DT_F32>(t, al, x, st);
    else bwd_t<DT_BF16>(t, al, x, st);
    return hipGetLastError();
}

}  // namespace lrscan
