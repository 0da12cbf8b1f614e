// delta_walk.hip -- gated delta rule: the walk over a sequence's blocks that
// carries a head's state, forward and back.
//
// One workgroup carries CT * 16 columns of one head's state [K, V] through all
// blocks of its batch row; the columns are independent.  A block's products follow
// one another,
//   K S -> X = (I + N)^-1 (V - enter K S) -> S' = end S + K^T (leave beta X),
// and each result becomes the next one's operand through LDS, cut into bf16
// planes there.  Four wavefronts do nothing but this chain; four more load the
// operands a block ahead, and take Q S and the outputs' product with U off it.
#include "delta_tile.hpp"
#include "delta_ws.hpp"

#include <type_traits>

namespace lrscan {
namespace delta {

constexpr int kTS = kC + 8;  // elements of an LDS column of 64 tokens

// Workgroups of one head lie on one XCD, so its q, k and rows of the inverse are
// read from memory once: bh % 8 is the workgroup's number % 8.
__device__ __forceinline__ bool my_head(const DeltaShape& s, int groups, int64_t& bh, int& group) {
    const int64_t r = blockIdx.x >> 3;
    group = (int)(r % groups);
    bh = r / groups * 8 + (blockIdx.x & 7);
    return bh < s.B * s.H;
}

// Eight wavefronts: `chain` ones (0 .. 3) carry the state, `side` ones (4 .. 7)
// bring the operands into LDS and do what does not wait for the state.  Of a
// block each has 16 tokens, of the state a chain wavefront 16 ND rows, all W columns.
constexpr int kWalkThreads = 512;
template <int RT, int CT>
struct Share {
    static constexpr int ND = RT;
    static constexpr int KP = 64 * RT, KS = KP + 8, W = CT * 16, VS = W + 8;
    static constexpr int kKPlane = kC * KS, kSPlane = W * KS, kTPlane = W * kTS;
};

// The block's gates, [3][kC] in LDS, brought by the first 64 side threads.
struct Gates {
    f32x4 x;
    __device__ __forceinline__ void load(const Prep& prep, int64_t t0, int len) {
        const uint32_t i = threadIdx.x & 255;
        x = __builtin_bit_cast(f32x4, load16(buffer(prep.gates + t0, len * 16), i < kC ? i * 16 : kNowhere));
    }
    __device__ __forceinline__ void store(float* lds) const {
        const int i = threadIdx.x & 255;
        if (i < kC) lds[i] = x[0], lds[kC + i] = x[1], lds[2 * kC + i] = x[2];
    }
};

// A tile of a block's kC rows and COLS columns, 8 columns a side thread at a time.
template <int DT, int COLS>
struct Tile {
    static constexpr int N = kC * COLS / 8, PER = (N + 255) / 256;
    Raw8<DT> x[PER];
    __device__ __forceinline__ void load(Buffer rows, int64_t st, int c0, int n) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = i * 256 + (threadIdx.x & 255);
            x[i].load(rows, o / (COLS / 8) * (int)st, c0 + o % (COLS / 8) * 8, n);
        }
    }
    __device__ __forceinline__ void store(uint16_t* tile, int plane, int stride) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = i * 256 + (threadIdx.x & 255);
            if (N % 256 == 0 || o < N) store_frag(tile + o / (COLS / 8) * stride + o % (COLS / 8) * 8, plane, x[i].frag());
        }
    }
};

// A wavefront's 16 rows of a contiguous [B, T, H, V] output, of which this
// workgroup has COLS columns: from accumulators through `lds` (the wavefront's
// own, 16 rows of COLS + 8 elements), in whole vectors or element by element.
template <int DT, int CT, bool WHOLE>
__device__ __forceinline__ void store_rows(void* out, char* lds, const DeltaShape& s, int64_t b, int h, int start, int len,
                                           int row0, int v0, const f32x4 (&x)[CT]) {
    constexpr int E = Elem<DT>::bytes, COLS = CT * 16, ROW = COLS + 8, PER = WHOLE ? 16 / E : 1, N = 16 * COLS / PER;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) put1<DT>(lds, ((lane >> 4) * 4 + r) * ROW + j * 16 + (lane & 15), x[j][r]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // one wavefront's LDS accesses keep their order
    const int64_t step = (int64_t)s.H * s.V * E;
    const Buffer rows = buffer(static_cast<char*>(out) + (b * s.T + start) * step + (int64_t)h * s.V * E, len * step);
#pragma unroll
    for (int i = 0; i < (N + 63) / 64; ++i) {
        const int o = i * 64 + lane, r = o / (COLS / PER), q = o % (COLS / PER) * PER;
        const bool ok = N % 64 == 0 || o < N;
        const uint32_t at = ok && v0 + q < s.V ? (row0 + r) * (int)step + (v0 + q) * E : kNowhere;
        const char* from = lds + ((ok ? r : 0) * ROW + q) * E;
        if constexpr (WHOLE)
            __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4*>(from), rows, at, 0, 0);
        else if constexpr (E == 4)
            __builtin_amdgcn_raw_buffer_store_b32(*reinterpret_cast<const uint32_t*>(from), rows, at, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(*reinterpret_cast<const uint16_t*>(from), rows, at, 0, 0);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// A chain wavefront's rows of a state scratch (rows of kw columns), and its
// tokens' rows of a token scratch; what lies past the rows or columns is left out.
template <int ND, int CT>
__device__ __forceinline__ void keep_state(float* to, const DeltaShape& s, int kw, int row0, int v0, int lane,
                                           const f32x4 (&x)[ND][CT]) {
    const Buffer rows = buffer(to, (int64_t)s.K * kw * 4);
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        const int col = v0 + j * 16 + (lane & 15);
        const uint32_t at = col < kw ? (uint32_t)(((row0 + (lane >> 4) * 4) * kw + col) * 4) : kNowhere;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) store4(rows, at, (i * 16 + r) * kw * 4, x[i][j][r]);
    }
}
template <int CT>
__device__ __forceinline__ void keep_tokens(float* to, int kw, int len, int row0, int v0, int lane, const f32x4 (&x)[CT]) {
    const Buffer rows = buffer(to, (int64_t)len * kw * 4);
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        const int col = v0 + j * 16 + (lane & 15);
        const uint32_t at = col < kw ? (uint32_t)(((row0 + (lane >> 4) * 4) * kw + col) * 4) : kNowhere;
#pragma unroll
        for (int r = 0; r < 4; ++r) store4(rows, at, r * kw * 4, x[j][r]);
    }
}

// A state [K, V] in or out of accumulators.
template <int ND, int CT, class F>
__device__ __forceinline__ void each_state(const DeltaShape& s, int64_t bh, int row0, int v0, int lane, F f) {
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = row0 + i * 16 + (lane >> 4) * 4 + r, col = v0 + j * 16 + (lane & 15);
                f(i, j, r, d < s.K && col < s.V, (bh * s.K + d) * s.V + col);
            }
}

// Elements of the operands' rows of K and of V.
struct Widths {
    int k, v;
};

template <int DT, int RT, int CT, bool KEEP, bool WHOLE>
__global__ void __launch_bounds__(kWalkThreads, DT == DT_BF16 && RT <= 2 ? 4 : 2)
delta_walk(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaFwd p, Kept keep, int groups, Widths wd) {
    using Sh = Share<RT, CT>;
    constexpr int NP = kPlanes<DT>, NA = kAttPlanes<DT>;
    constexpr int ND = Sh::ND, KP = Sh::KP, KS = Sh::KS, W = Sh::W, VS = Sh::VS;
    constexpr int kKPlane = Sh::kKPlane, kSPlane = Sh::kSPlane, kTPlane = Sh::kTPlane;
    constexpr int kU = KEEP ? 0 : NA;  // planes of u beside the three of leave u
    constexpr int kWide = 3 * kSPlane > (kU + 3) * kTPlane ? 3 * kSPlane : (kU + 3) * kTPlane;
    __shared__ __attribute__((aligned(16))) uint16_t kt[NP * kKPlane];  // K of the block [token][row]
    __shared__ __attribute__((aligned(16))) uint16_t wide[kWide];       // the state, then u and leave u
    __shared__ __attribute__((aligned(16))) uint16_t rt[3 * kTPlane];   // right sides of the triangular system
    __shared__ __attribute__((aligned(16))) uint16_t vt[NP * kC * VS];  // V [token][column]
    __shared__ __attribute__((aligned(16))) char ot[KEEP ? 16 : kC * VS * Elem<DT>::bytes];  // the outputs, as stored
    __shared__ __attribute__((aligned(16))) float gates[3 * kC];
    uint16_t *const ut = wide, *const lt = wide + kU * kTPlane;

    int64_t bh;
    int group;
    if (!my_head(s, groups, bh, group)) return;
    const int64_t b = bh / s.H;
    const int h = (int)(bh % s.H), hk = h / (s.H / s.HK);
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int v0 = group * W, wr = w & 3;
    const int row0 = wr * 16, r0 = row0 + lg * 4;  // tokens of the wavefront, and of the lane in a tile of results
    const int n = blocks.count(b);
    int start, len;
    bool cut;
    blocks.at(b, 0, start, len, cut);

    if (w < 4) {
        const int d0 = wr * ND * 16, kw = kept_width(s.V);
        f32x4 S[ND][CT];
        each_state<ND, CT>(s, bh, d0, v0, lane,
                           [&](int i, int j, int r, bool ok, int64_t at) { S[i][j][r] = in.h0 && ok ? in.h0[at] : 0.0f; });
        Frag<3> ti[2];
        // tokens of the lower half of a block reach its first 32 only
        auto load_inv = [&](int start, int len) {
            const Buffer rows = plane_rows<3>(prep.inv, bh * s.T + start, len);
            ti[0] = plane_frag<3>(rows, row0 + ln, lg * 8);
            if (wr >= 2) ti[1] = plane_frag<3>(rows, row0 + ln, 32 + lg * 8);
        };
        load_inv(start, len);
        for (int c = 0; c < n; ++c) {
            // the next block; past the last one, one without tokens
            int next = s.T, nlen = 0;
            bool ncut = false;
            if (c + 1 < n) blocks.at(b, c + 1, next, nlen, ncut);
            if (cut) {
#pragma unroll
                for (int i = 0; i < ND; ++i)
#pragma unroll
                    for (int j = 0; j < CT; ++j) S[i][j] = f32x4{0, 0, 0, 0};
            } else if (KEEP) {
                keep_state<ND, CT>(keep.s + (bh * state_slots(s.T) + start / kC) * s.K * kw, s, kw, d0, v0, lane, S);
            }
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    store_planes(wide + (j * 16 + ln) * KS + d0 + i * 16 + lg * 4, kSPlane, S[i][j]);
            __syncthreads();  // the operands and the state are in LDS

            f32x4 ks[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) ks[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KP; k += 32) {
                Frag<3> sf[CT];
#pragma unroll
                for (int j = 0; j < CT; ++j) sf[j] = row_frag<3>(wide, kSPlane, KS, j * 16, k, lane);
                mma(ks, row_frag<NP>(kt, kKPlane, KS, row0, k, lane), sf);
            }
            const f32x4 en = *reinterpret_cast<const f32x4*>(gates + r0);
            const f32x4 le = *reinterpret_cast<const f32x4*>(gates + kC + r0);
            const f32x4 be = *reinterpret_cast<const f32x4*>(gates + 2 * kC + r0);
            const float end = gates[len - 1];
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                f32x4 y;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    y[r] = fmaf(-en[r], ks[j][r], element<NP>(vt + (r0 + r) * VS + j * 16 + ln, kC * VS));
                store_planes(rt + (j * 16 + ln) * kTS + r0, kTPlane, y);
            }
            __syncthreads();  // the right sides are

            f32x4 x[CT];
            Frag<3> f[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                x[j] = f32x4{0, 0, 0, 0};
                f[j] = row_frag<3>(rt, kTPlane, kTS, j * 16, 0, lane);
            }
            mma(x, ti[0], f);
            if (wr >= 2) {
#pragma unroll
                for (int j = 0; j < CT; ++j) f[j] = row_frag<3>(rt, kTPlane, kTS, j * 16, 32, lane);
                mma(x, ti[1], f);
            }
            load_inv(next, nlen);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                f32x4 u, l;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    u[r] = be[r] * x[j][r];
                    l[r] = le[r] * u[r];
                }
                const int o = (j * 16 + ln) * kTS + r0;
                if (!KEEP) store_planes<NA>(ut + o, kTPlane, u);
                store_planes(lt + o, kTPlane, l);
            }
            __syncthreads();  // u is

            if (KEEP) keep_tokens<CT>(keep.x + (bh * s.T + start) * kw, kw, len, row0, v0, lane, x);
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[i][j][r] *= end;
#pragma unroll
            for (int k = 0; k < kC; k += 32) {
#pragma unroll
                for (int j = 0; j < CT; ++j) f[j] = row_frag<3>(lt, kTPlane, kTS, j * 16, k, lane);
#pragma unroll
                for (int i = 0; i < ND; ++i) mma(S[i], col_frag<NP>(kt, kKPlane, KS, k, d0 + i * 16, lane), f);
            }
            __syncthreads();  // and all of it is read
            start = next, len = nlen, cut = ncut;
        }
        if (!KEEP && p.last)
            each_state<ND, CT>(s, bh, d0, v0, lane, [&](int i, int j, int r, bool ok, int64_t at) {
                if (ok) p.last[at] = S[i][j][r];
            });
        return;
    }

    Tile<DT, KP> kn;
    Tile<DT, W> vn;
    Gates gn;
    Raw8<DT> qn[KP / 32];
    Frag<NA> at[2];
    auto load = [&](int start, int len) {
        kn.load(block_rows(in.k, b, hk, start, len), in.k.st, 0, wd.k);
        vn.load(block_rows(in.v, b, h, start, len), in.v.st, v0, wd.v);
        gn.load(prep, bh * s.T + start, len);
    };
    auto load_q = [&](int start, int len) {
        const Buffer rows = block_rows(in.q, b, hk, start, len);
#pragma unroll
        for (int k = 0; k < KP / 32; ++k) qn[k].load(rows, (row0 + ln) * (int)in.q.st, k * 32 + lg * 8, wd.k);
    };
    auto load_att = [&](int start, int len) {
        const Buffer rows = plane_rows<NA>(prep.att, bh * s.T + start, len);
        at[0] = plane_frag<NA>(rows, row0 + ln, lg * 8);
        if (wr >= 2) at[1] = plane_frag<NA>(rows, row0 + ln, 32 + lg * 8);
    };
    load(start, len);
    if (!KEEP) {
        load_q(start, len);
        load_att(start, len);
    }
    for (int c = 0; c < n; ++c) {
        int next = s.T, nlen = 0;
        if (c + 1 < n) blocks.at(b, c + 1, next, nlen, cut);
        kn.store(kt, kKPlane, KS);
        vn.store(vt, kC * VS, VS);
        gn.store(gates);
        __syncthreads();
        load(next, nlen);
        f32x4 qs[CT], o[CT];
        if (!KEEP) {
#pragma unroll
            for (int j = 0; j < CT; ++j) qs[j] = o[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KP / 32; ++k) {
                Frag<NA> sf[CT];
#pragma unroll
                for (int j = 0; j < CT; ++j) sf[j] = row_frag<NA>(wide, kSPlane, KS, j * 16, k * 32, lane);
                mma(qs, qn[k].frag(), sf);
            }
            load_q(next, nlen);
            const f32x4 en = *reinterpret_cast<const f32x4*>(gates + r0);
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) qs[j][r] *= en[r];
        }
        __syncthreads();
        __syncthreads();
        if (!KEEP) {
            Frag<NA> f[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) f[j] = row_frag<NA>(ut, kTPlane, kTS, j * 16, 0, lane);
            mma(o, at[0], f);
            if (wr >= 2) {
#pragma unroll
                for (int j = 0; j < CT; ++j) f[j] = row_frag<NA>(ut, kTPlane, kTS, j * 16, 32, lane);
                mma(o, at[1], f);
            }
            load_att(next, nlen);
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[j][r] = in.scale * (qs[j][r] + o[j][r]);
            if (p.out)
                store_rows<DT, CT, WHOLE>(p.out, ot + row0 * VS * Elem<DT>::bytes, s, b, h, start, len, row0, v0, o);
        }
        __syncthreads();
        start = next, len = nlen;
    }
}

// The walk back.  With P the outputs' weights, dS the gradient of the state
// that leaves a block and everything scaled as above,
//   dU = scale P^T dO + leave K dS,  R = (I + diag(beta) M)^-T dU  (the gradient
//   of beta (V - enter K S)),  dV = beta R,
//   dS' = end dS + Q^T (scale enter dO) - K^T (beta enter R).
template <int DT, int RT, int CT, bool WHOLE>
__global__ void __launch_bounds__(kWalkThreads, DT == DT_BF16 && RT == 1 ? 4 : 2)
delta_walk_back(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaBwd p, HeadRows go, Kept keep, int groups,
                Widths wd) {
    using Sh = Share<RT, CT>;
    constexpr int NP = kPlanes<DT>;
    constexpr int ND = Sh::ND, KP = Sh::KP, KS = Sh::KS, W = Sh::W, VS = Sh::VS;
    constexpr int kKPlane = Sh::kKPlane, kSPlane = Sh::kSPlane, kTPlane = Sh::kTPlane, kOPlane = kC * VS;
    constexpr int kWide = 3 * (kSPlane > 2 * kTPlane ? kSPlane : 2 * kTPlane);
    // fp32 tiles of K and Q together pass the LDS from 65 rows on: Q then takes K's place
    constexpr bool kShare = DT == DT_F32 && RT >= 2;
    __shared__ __attribute__((aligned(16))) uint16_t kt[NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t qt_[kShare ? 8 : NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t wide[kWide];  // dS, then what goes into K^T and Q^T
    __shared__ __attribute__((aligned(16))) uint16_t rt[3 * kTPlane];
    __shared__ __attribute__((aligned(16))) uint16_t ot[NP * kOPlane];  // dO [token][column]
    __shared__ __attribute__((aligned(16))) char gt[kC * VS * Elem<DT>::bytes];  // dV, as stored
    __shared__ __attribute__((aligned(16))) float gates[3 * kC];
    uint16_t *const lt = wide, *const et = wide + 3 * kTPlane;
    uint16_t* const qt = kShare ? kt : qt_;

    int64_t bh;
    int group;
    if (!my_head(s, groups, bh, group)) return;
    const int64_t b = bh / s.H;
    const int h = (int)(bh % s.H), hk = h / (s.H / s.HK);
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int v0 = group * W, wr = w & 3;
    const int row0 = wr * 16, r0 = row0 + lg * 4;
    const int64_t slots = state_slots(s.T);
    const int n = blocks.count(b);
    int start, len;
    bool first;  // whether a segment starts with the block
    blocks.at(b, n - 1, start, len, first);

    if (w < 4) {
        const int d0 = wr * ND * 16, kw = kept_width(s.V);
        f32x4 S[ND][CT];
        each_state<ND, CT>(s, bh, d0, v0, lane, [&](int i, int j, int r, bool ok, int64_t at) {
            S[i][j][r] = p.grad_last && ok ? p.grad_last[at] : 0.0f;
        });
        Frag<3> ti[2], at[2];  // columns of the inverse and of the weights: tokens from a row's own on
        auto load_cols = [&](Frag<3> (&f)[2], const uint16_t* p, int start, int len) {
            const Buffer rows = plane_rows<3>(p, bh * s.T + start, len);
            if (wr < 2) f[0] = plane_frag<3>(rows, row0 + ln, lg * 8);
            f[1] = plane_frag<3>(rows, row0 + ln, 32 + lg * 8);
        };
        load_cols(at, prep.att_t, start, len);
        load_cols(ti, prep.inv_t, start, len);
        // what leaves a block enters the one behind it, unless a segment starts there
        bool cut = false;
        for (int c = n - 1; c >= 0; --c) {
            const int behind = start + len;
            int prev = 0, plen = 0;
            bool pfirst = false;
            if (c > 0) blocks.at(b, c - 1, prev, plen, pfirst);
            if (cut) {
#pragma unroll
                for (int i = 0; i < ND; ++i)
#pragma unroll
                    for (int j = 0; j < CT; ++j) S[i][j] = f32x4{0, 0, 0, 0};
            } else {
                keep_state<ND, CT>(keep.ds + (bh * slots + (behind < s.T ? behind / kC : slots - 1)) * s.K * kw, s, kw, d0,
                                   v0, lane, S);
            }
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    store_planes(wide + (j * 16 + ln) * KS + d0 + i * 16 + lg * 4, kSPlane, S[i][j]);
            __syncthreads();  // the operands and dS are in LDS

            f32x4 kd[CT], po[CT];
            Frag<NP> of[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) kd[j] = po[j] = f32x4{0, 0, 0, 0};
            if (wr < 2) {
#pragma unroll
                for (int j = 0; j < CT; ++j) of[j] = col_frag<NP>(ot, kOPlane, VS, 0, j * 16, lane);
                mma(po, at[0], of);
            }
#pragma unroll
            for (int j = 0; j < CT; ++j) of[j] = col_frag<NP>(ot, kOPlane, VS, 32, j * 16, lane);
            mma(po, at[1], of);
            load_cols(at, prep.att_t, prev, plen);
            Frag<3> f[CT];
#pragma unroll
            for (int k = 0; k < KP; k += 32) {
#pragma unroll
                for (int j = 0; j < CT; ++j) f[j] = row_frag<3>(wide, kSPlane, KS, j * 16, k, lane);
                mma(kd, row_frag<NP>(kt, kKPlane, KS, row0, k, lane), f);
            }
            const f32x4 en = *reinterpret_cast<const f32x4*>(gates + r0);
            const f32x4 le = *reinterpret_cast<const f32x4*>(gates + kC + r0);
            const f32x4 be = *reinterpret_cast<const f32x4*>(gates + 2 * kC + r0);
            const float end = gates[len - 1];
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                f32x4 y;
#pragma unroll
                for (int r = 0; r < 4; ++r) y[r] = fmaf(le[r], kd[j][r], in.scale * po[j][r]);
                store_planes(rt + (j * 16 + ln) * kTS + r0, kTPlane, y);
            }
            __syncthreads();  // dU is

            f32x4 x[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) x[j] = f32x4{0, 0, 0, 0};
            if (wr < 2) {
#pragma unroll
                for (int j = 0; j < CT; ++j) f[j] = row_frag<3>(rt, kTPlane, kTS, j * 16, 0, lane);
                mma(x, ti[0], f);
            }
#pragma unroll
            for (int j = 0; j < CT; ++j) f[j] = row_frag<3>(rt, kTPlane, kTS, j * 16, 32, lane);
            mma(x, ti[1], f);
            load_cols(ti, prep.inv_t, prev, plen);
            f32x4 dv[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                f32x4 l;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dv[j][r] = be[r] * x[j][r];
                    l[r] = -en[r] * dv[j][r];
                }
                store_planes(lt + (j * 16 + ln) * kTS + r0, kTPlane, l);
            }
            __syncthreads();  // what goes into K^T and Q^T is

            keep_tokens<CT>(keep.r + (bh * s.T + start) * kw, kw, len, row0, v0, lane, x);
            store_rows<DT, CT, WHOLE>(p.grad_v, gt + row0 * VS * Elem<DT>::bytes, s, b, h, start, len, row0, v0, dv);
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[i][j][r] *= end;
#pragma unroll
            for (int k = 0; k < kC; k += 32) {
#pragma unroll
                for (int j = 0; j < CT; ++j) f[j] = row_frag<3>(lt, kTPlane, kTS, j * 16, k, lane);
#pragma unroll
                for (int i = 0; i < ND; ++i) mma(S[i], col_frag<NP>(kt, kKPlane, KS, k, d0 + i * 16, lane), f);
            }
            if (kShare) {
                __syncthreads();  // K is read
                __syncthreads();  // Q is in its place
            }
#pragma unroll
            for (int k = 0; k < kC; k += 32) {
#pragma unroll
                for (int j = 0; j < CT; ++j) f[j] = row_frag<3>(et, kTPlane, kTS, j * 16, k, lane);
#pragma unroll
                for (int i = 0; i < ND; ++i) mma(S[i], col_frag<NP>(qt, kKPlane, KS, k, d0 + i * 16, lane), f);
            }
            __syncthreads();  // and all of it is read
            start = prev, len = plen, cut = first, first = pfirst;
        }
        if (p.grad_h0)
            each_state<ND, CT>(s, bh, d0, v0, lane, [&](int i, int j, int r, bool ok, int64_t at) {
                if (ok) p.grad_h0[at] = cut ? 0.0f : S[i][j][r];
            });
        return;
    }

    Tile<DT, KP> kn, qn;
    Tile<DT, W> on;
    Gates gn;
    auto load = [&](int start, int len) {
        kn.load(block_rows(in.k, b, hk, start, len), in.k.st, 0, wd.k);
        if (!kShare) qn.load(block_rows(in.q, b, hk, start, len), in.q.st, 0, wd.k);
        on.load(block_rows(go, b, h, start, len), go.st, v0, wd.v);
        gn.load(prep, bh * s.T + start, len);
    };
    load(start, len);
    for (int c = n - 1; c >= 0; --c) {
        int prev = 0, plen = 0;
        if (c > 0) blocks.at(b, c - 1, prev, plen, first);
        kn.store(kt, kKPlane, KS);
        if (!kShare) qn.store(qt, kKPlane, KS);
        on.store(ot, kOPlane, VS);
        gn.store(gates);
        __syncthreads();
        if (kShare) qn.load(block_rows(in.q, b, hk, start, len), in.q.st, 0, wd.k);
        load(prev, plen);
        const f32x4 en = *reinterpret_cast<const f32x4*>(gates + r0);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            f32x4 e;
#pragma unroll
            for (int r = 0; r < 4; ++r) e[r] = in.scale * en[r] * element<NP>(ot + (r0 + r) * VS + j * 16 + ln, kOPlane);
            store_planes(et + (j * 16 + ln) * kTS + r0, kTPlane, e);
        }
        __syncthreads();
        if (kShare) {
            __syncthreads();
            qn.store(qt, kKPlane, KS);
            __syncthreads();
        }
        __syncthreads();
        start = prev, len = plen;
    }
}

// Columns of a workgroup: 32, or 16 where fp32 tiles of K leave no room for
// more, or where V has no more.
template <int DT, int RT>
constexpr int kMaxCT = DT == DT_F32 && RT >= 3 ? 1 : 2;

template <class F>
hipError_t by_rows(const DeltaShape& s, F f) {
    switch ((s.K + 63) / 64) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        default: return f(std::integral_constant<int, 4>{});
    }
}

// Whether rows of a [B, T, H, V] output are whole aligned vectors.
bool whole(const DeltaShape& s, const void* p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(s.V * (dtype == DT_F32 ? 4 : 2))) % 16 == 0;
}

dim3 walk_grid(const DeltaShape& s, int groups) { return dim3((unsigned)((s.B * s.H + 7) / 8 * 8 * groups)); }

template <int DT, bool KEEP>
hipError_t walk(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaFwd& out,
                const Kept& keep, hipStream_t st) {
    const Widths wd{row_width(s.K, DT), row_width(s.V, DT)};
    const bool rows = whole(s, out.out, DT);
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, CT = kMaxCT<DT, RT>;
        const int groups = (s.V + CT * 16 - 1) / (CT * 16);
        if (KEEP || rows)
            delta_walk<DT, RT, CT, KEEP, true><<<walk_grid(s, groups), kWalkThreads, 0, st>>>(s, in, blocks, prep, out, keep, groups, wd);
        else
            delta_walk<DT, RT, CT, KEEP, KEEP><<<walk_grid(s, groups), kWalkThreads, 0, st>>>(s, in, blocks, prep, out, keep, groups, wd);
        return hipGetLastError();
    });
}

hipError_t run_walk(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                    const DeltaFwd& out, const Kept* keep, hipStream_t st) {
    if (s.dtype == DT_BF16)
        return keep ? walk<DT_BF16, true>(s, in, blocks, prep, out, *keep, st)
                    : walk<DT_BF16, false>(s, in, blocks, prep, out, Kept{}, st);
    return keep ? walk<DT_F32, true>(s, in, blocks, prep, out, *keep, st)
                : walk<DT_F32, false>(s, in, blocks, prep, out, Kept{}, st);
}

template <int DT>
hipError_t walk_back(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaBwd& p,
                     const HeadRows& go, const Kept& keep, hipStream_t st) {
    const Widths wd{row_width(s.K, DT), row_width(s.V, DT)};
    const bool rows = whole(s, p.grad_v, DT);
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, CT = kMaxCT<DT, RT>;
        const int groups = (s.V + CT * 16 - 1) / (CT * 16);
        if (rows)
            delta_walk_back<DT, RT, CT, true><<<walk_grid(s, groups), kWalkThreads, 0, st>>>(s, in, blocks, prep, p, go, keep, groups, wd);
        else
            delta_walk_back<DT, RT, CT, false><<<walk_grid(s, groups), kWalkThreads, 0, st>>>(s, in, blocks, prep, p, go, keep, groups, wd);
        return hipGetLastError();
    });
}

hipError_t run_walk_back(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                         const DeltaBwd& p, const HeadRows& go, const Kept& keep, hipStream_t st) {
    return s.dtype == DT_BF16 ? walk_back<DT_BF16>(s, in, blocks, prep, p, go, keep, st)
                              : walk_back<DT_F32>(s, in, blocks, prep, p, go, keep, st);
}

}  // namespace delta
}  // namespace lrscan
