// delta_walk.hip -- gated delta rule: the walk over a sequence's blocks that
// carries a head's state, forward and back.
//
// One workgroup carries CT * 16 columns of one head's state [K, V] through all
// blocks of its batch row; the columns are independent.  Its four wavefronts
// share the columns' tiles of 16 and, of those, the state's rows (held in
// accumulators) and the block's tokens.  A block's products follow one another,
//   K S -> X = (I + N)^-1 (V - enter K S) -> S' = end S + K^T (leave beta X),
// and each result becomes the next one's operand through LDS, cut into bf16
// planes there.  Q S and the outputs' product with U fill in beside them.  What
// the next block reads from memory is loaded into registers a block ahead, each
// operand as soon as this block's is used.
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

// What a workgroup's wavefronts have of a block: of W columns the tile wc, of the
// tokens NT tiles of 16 from wr NT on, of the state's rows ND from wr ND on.
template <int RT, int CT>
struct Share {
    static constexpr int WR = 4 / CT, NT = 4 / WR, ND = 4 * RT / WR;
    static constexpr int KP = 64 * RT, KS = KP + 8, W = CT * 16, VS = W + 8;
    static constexpr int kKPlane = kC * KS, kSPlane = W * KS, kTPlane = W * kTS;
};

// The block's gates, [3][kC] in LDS; a thread of the first 64 loads its token's.
struct Gates {
    float enter, leave, beta;
    __device__ __forceinline__ void load(const DeltaIn& in, const Prep& prep, int64_t b, int64_t h, int64_t t0, int start,
                                         int len) {
        enter = leave = beta = 0.0f;
        const int i = threadIdx.x;
        if (i < len) {
            enter = prep.enter[t0 + i];
            leave = prep.leave[t0 + i];
            beta = *reinterpret_cast<const float*>(in.beta.row(b, start + i, h));
        }
    }
    __device__ __forceinline__ void store(float* lds) const {
        if (threadIdx.x < kC) lds[threadIdx.x] = enter, lds[kC + threadIdx.x] = leave, lds[2 * kC + threadIdx.x] = beta;
    }
};

// A tile of a block's kC rows and COLS columns, 8 columns a thread at a time.
template <int DT, int COLS>
struct Tile {
    static constexpr int N = kC * COLS / 8, PER = (N + kThreads - 1) / kThreads;
    Raw8<DT> x[PER];
    __device__ __forceinline__ void load(Buffer rows, int64_t st, int c0, int n) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = i * kThreads + threadIdx.x;
            x[i].load(rows, o / (COLS / 8) * (int)st, c0 + o % (COLS / 8) * 8, n);
        }
    }
    __device__ __forceinline__ void store(uint16_t* tile, int plane, int stride) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = i * kThreads + threadIdx.x;
            if (N % kThreads == 0 || o < N) store_frag(tile + o / (COLS / 8) * stride + o % (COLS / 8) * 8, plane, x[i].frag());
        }
    }
};

// Rows of an [.., H, V] output from LDS elements [kC][stride], 8 columns a thread.
template <int DT, int COLS>
__device__ __forceinline__ void store_rows(void* out, const char* lds, int stride, const DeltaShape& s, int64_t b, int h,
                                           int start, int len, int v0, bool vec) {
    constexpr int N = kC * COLS / 8, E = Elem<DT>::bytes;
    for (int o = threadIdx.x; o < N; o += kThreads) {
        const int r = o / (COLS / 8), q = o % (COLS / 8) * 8;
        if (r >= len || v0 + q >= s.V) continue;
        const char* from = lds + (r * stride + q) * E;
        char* to = static_cast<char*>(out) + (((b * s.T + start + r) * s.H + h) * (int64_t)s.V + v0 + q) * E;
        if (vec) {
            *reinterpret_cast<u32x4*>(to) = *reinterpret_cast<const u32x4*>(from);
            if (E == 4 && v0 + q + 4 < s.V) *reinterpret_cast<u32x4*>(to + 16) = *reinterpret_cast<const u32x4*>(from + 16);
        } else {
            for (int j = 0; j < 8 && v0 + q + j < s.V; ++j) {
                if (E == 4)
                    reinterpret_cast<uint32_t*>(to)[j] = reinterpret_cast<const uint32_t*>(from)[j];
                else
                    reinterpret_cast<uint16_t*>(to)[j] = reinterpret_cast<const uint16_t*>(from)[j];
            }
        }
    }
}

// Elements of the operands' rows of K and of V, and whether rows of the output are whole vectors.
struct Widths {
    int k, v;
    bool out;
};

template <int DT, int RT, int CT, bool KEEP>
__global__ void __launch_bounds__(kThreads, DT == DT_BF16 && RT <= 2 ? 2 : 1)
delta_walk(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaFwd p, Kept keep, int groups, Widths wd) {
    using Sh = Share<RT, CT>;
    constexpr int NP = kPlanes<DT>, NA = kAttPlanes<DT>;
    constexpr int NT = Sh::NT, ND = Sh::ND, KP = Sh::KP, KS = Sh::KS, W = Sh::W, VS = Sh::VS;
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
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, ln = lane & 15, lg = lane >> 4;
    const int wc = w % CT, wr = w / CT;
    const int v0 = group * W, col = v0 + wc * 16 + ln;

    f32x4 S[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = (wr * ND + i) * 16 + lg * 4 + r;
            S[i][r] = in.h0 && d < s.K && col < s.V ? in.h0[(bh * s.K + d) * s.V + col] : 0.0f;
        }

    // rows of kw columns, of which this lane has one; what lies past the state's rows or columns is left out
    const int kw = kept_width(s.V);
    const uint32_t kept_at = col < kw ? (uint32_t)(((wr * ND * 16 + lg * 4) * kw + col) * 4) : kNowhere;
    auto keep_state = [&](float* to, const f32x4 (&x)[ND]) {
        const Buffer rows = buffer(to, (int64_t)s.K * kw * 4);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) store4(rows, kept_at, (i * 16 + r) * kw * 4, x[i][r]);
    };
    const uint32_t kept_x = col < kw ? (uint32_t)(((wr * NT * 16 + lg * 4) * kw + col) * 4) : kNowhere;
    auto keep_tokens = [&](float* to, int start, int len, const f32x4 (&x)[NT]) {
        const Buffer rows = buffer(to + (bh * s.T + start) * kw, (int64_t)len * kw * 4);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) store4(rows, kept_x, (i * 16 + r) * kw * 4, x[i][r]);
    };

    Tile<DT, KP> kn;
    Tile<DT, W> vn;
    Raw8<DT> qn[NT][KP / 32];
    Frag<3> ti[NT][2];
    Frag<NA> at[NT][2];
    Gates gn;
    auto token = [&](int i) { return (wr * NT + i) * 16 + ln; };
    auto load_q = [&](int start, int len) {
        const Buffer rows = block_rows(in.q, b, hk, start, len);
        if (!KEEP)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < KP / 32; ++k)
                    qn[i][k].load(rows, token(i) * (int)in.q.st, k * 32 + lg * 8, wd.k);
    };
    // tokens of the lower half of a block reach its first 32 only
    auto load_inv = [&](int start, int len) {
        const Buffer rows = plane_rows<3>(prep.inv, bh * s.T + start, len);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k == 0 || wr * NT + i >= 2) ti[i][k] = plane_frag<3>(rows, token(i), k * 32 + lg * 8);
    };
    auto load_att = [&](int start, int len) {
        const Buffer rows = plane_rows<NA>(prep.att, bh * s.T + start, len);
        if (!KEEP)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (k == 0 || wr * NT + i >= 2) at[i][k] = plane_frag<NA>(rows, token(i), k * 32 + lg * 8);
    };

    const int n = blocks.count(b);
    int start, len;
    bool cut;
    blocks.at(b, 0, start, len, cut);
    kn.load(block_rows(in.k, b, hk, start, len), in.k.st, 0, wd.k);
    vn.load(block_rows(in.v, b, h, start, len), in.v.st, v0, wd.v);
    gn.load(in, prep, b, h, bh * s.T + start, start, len);
    load_q(start, len);
    load_inv(start, len);
    load_att(start, len);
    for (int c = 0; c < n; ++c) {
        // the next block; past the last one, one without tokens
        int next = s.T, nlen = 0;
        bool ncut = false;
        if (c + 1 < n) blocks.at(b, c + 1, next, nlen, ncut);
        if (cut) {
#pragma unroll
            for (int i = 0; i < ND; ++i) S[i] = f32x4{0, 0, 0, 0};
        } else if (KEEP) {
            keep_state(keep.s + (bh * state_slots(s.T) + start / kC) * s.K * kw, S);
        }
        kn.store(kt, kKPlane, KS);
        vn.store(vt, kC * VS, VS);
        gn.store(gates);
#pragma unroll
        for (int i = 0; i < ND; ++i)
            store_planes(wide + (wc * 16 + ln) * KS + (wr * ND + i) * 16 + lg * 4, kSPlane, S[i]);
        __syncthreads();
        kn.load(block_rows(in.k, b, hk, next, nlen), in.k.st, 0, wd.k);
        vn.load(block_rows(in.v, b, h, next, nlen), in.v.st, v0, wd.v);
        gn.load(in, prep, b, h, bh * s.T + next, next, nlen);

        f32x4 ks_[NT], qs[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) ks_[i] = qs[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KP / 32; ++k) {
            const Frag<3> sf = row_frag<3>(wide, kSPlane, KS, wc * 16, k * 32, lane);
            Frag<NA> sa;
#pragma unroll
            for (int i = 0; i < NA; ++i) sa.p[i] = sf.p[i];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                mma(ks_[i], row_frag<NP>(kt, kKPlane, KS, (wr * NT + i) * 16, k * 32, lane), sf);
                if (!KEEP) mma(qs[i], qn[i][k].frag(), sa);
            }
        }
        load_q(next, nlen);
        f32x4 en[NT], le[NT], be[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r0 = (wr * NT + i) * 16 + lg * 4;
            en[i] = *reinterpret_cast<const f32x4*>(gates + r0);
            le[i] = *reinterpret_cast<const f32x4*>(gates + kC + r0);
            be[i] = *reinterpret_cast<const f32x4*>(gates + 2 * kC + r0);
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y[r] = fmaf(-en[i][r], ks_[i][r], element<NP>(vt + (r0 + r) * VS + wc * 16 + ln, kC * VS));
            store_planes(rt + (wc * 16 + ln) * kTS + r0, kTPlane, y);
        }
        const float end = gates[len - 1];
        __syncthreads();

        f32x4 x[NT];
        {
            const Frag<3> y0 = row_frag<3>(rt, kTPlane, kTS, wc * 16, 0, lane);
            const Frag<3> y1 = row_frag<3>(rt, kTPlane, kTS, wc * 16, 32, lane);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                x[i] = f32x4{0, 0, 0, 0};
                mma(x[i], ti[i][0], y0);
                if (wr * NT + i >= 2) mma(x[i], ti[i][1], y1);
            }
        }
        load_inv(next, nlen);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int at_ = (wc * 16 + ln) * kTS + (wr * NT + i) * 16 + lg * 4;
            f32x4 u, l;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                u[r] = be[i][r] * x[i][r];
                l[r] = le[i][r] * u[r];
            }
            if (!KEEP) store_planes<NA>(ut + at_, kTPlane, u);
            store_planes(lt + at_, kTPlane, l);
        }
        __syncthreads();

        if (KEEP) {
            keep_tokens(keep.x, start, len, x);
        } else {
            const Frag<NA> u0 = row_frag<NA>(ut, kTPlane, kTS, wc * 16, 0, lane);
            const Frag<NA> u1 = row_frag<NA>(ut, kTPlane, kTS, wc * 16, 32, lane);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                f32x4 o = {0, 0, 0, 0};
                mma(o, at[i][0], u0);
                if (wr * NT + i >= 2) mma(o, at[i][1], u1);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    put1<DT>(ot, ((wr * NT + i) * 16 + lg * 4 + r) * VS + wc * 16 + ln,
                             in.scale * fmaf(en[i][r], qs[i][r], o[r]));
            }
        }
        load_att(next, nlen);
        {
            const Frag<3> l0 = row_frag<3>(lt, kTPlane, kTS, wc * 16, 0, lane);
            const Frag<3> l1 = row_frag<3>(lt, kTPlane, kTS, wc * 16, 32, lane);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] *= end;
                mma(S[i], col_frag<NP>(kt, kKPlane, KS, 0, (wr * ND + i) * 16, lane), l0);
                mma(S[i], col_frag<NP>(kt, kKPlane, KS, 32, (wr * ND + i) * 16, lane), l1);
            }
        }
        __syncthreads();
        if (!KEEP && p.out) store_rows<DT, W>(p.out, ot, VS, s, b, h, start, len, v0, wd.out);
        start = next, len = nlen, cut = ncut;
    }
    if (!KEEP && p.last)
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = (wr * ND + i) * 16 + lg * 4 + r;
                if (d < s.K && col < s.V) p.last[(bh * s.K + d) * s.V + col] = S[i][r];
            }
}

// The walk back.  With P the outputs' weights, dS the gradient of the state
// that leaves a block and everything scaled as above,
//   dU = scale P^T dO + leave K dS,  R = (I + diag(beta) M)^-T dU  (the gradient
//   of beta (V - enter K S)),  dV = beta R,
//   dS' = end dS + Q^T (scale enter dO) - K^T (beta enter R).
template <int DT, int RT, int CT>
__global__ void __launch_bounds__(kThreads, DT == DT_BF16 && RT == 1 ? 2 : 1)
delta_walk_back(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaBwd p, HeadRows go, Kept keep,
                int groups, Widths wd) {
    using Sh = Share<RT, CT>;
    constexpr int NP = kPlanes<DT>;
    constexpr int NT = Sh::NT, ND = Sh::ND, KP = Sh::KP, KS = Sh::KS, W = Sh::W, VS = Sh::VS;
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
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, ln = lane & 15, lg = lane >> 4;
    const int wc = w % CT, wr = w / CT;
    const int v0 = group * W, col = v0 + wc * 16 + ln;
    const int64_t slots = state_slots(s.T);

    f32x4 S[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = (wr * ND + i) * 16 + lg * 4 + r;
            S[i][r] = p.grad_last && d < s.K && col < s.V ? p.grad_last[(bh * s.K + d) * s.V + col] : 0.0f;
        }

    // rows of kw columns, of which this lane has one; what lies past the state's rows or columns is left out
    const int kw = kept_width(s.V);
    const uint32_t kept_at = col < kw ? (uint32_t)(((wr * ND * 16 + lg * 4) * kw + col) * 4) : kNowhere;
    auto keep_state = [&](float* to, const f32x4 (&x)[ND]) {
        const Buffer rows = buffer(to, (int64_t)s.K * kw * 4);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) store4(rows, kept_at, (i * 16 + r) * kw * 4, x[i][r]);
    };
    const uint32_t kept_x = col < kw ? (uint32_t)(((wr * NT * 16 + lg * 4) * kw + col) * 4) : kNowhere;
    auto keep_tokens = [&](float* to, int start, int len, const f32x4 (&x)[NT]) {
        const Buffer rows = buffer(to + (bh * s.T + start) * kw, (int64_t)len * kw * 4);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) store4(rows, kept_x, (i * 16 + r) * kw * 4, x[i][r]);
    };

    Tile<DT, KP> kn, qn;
    Tile<DT, W> on;
    Frag<3> ti[NT][2], at[NT][2];  // columns of the inverse and of the weights: tokens from a row's own on
    Gates gn;
    auto load_cols = [&](Frag<3> (&f)[NT][2], const uint16_t* p, int start, int len) {
        const Buffer rows = plane_rows<3>(p, bh * s.T + start, len);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k == 1 || wr * NT + i < 2) f[i][k] = plane_frag<3>(rows, (wr * NT + i) * 16 + ln, k * 32 + lg * 8);
    };

    const int n = blocks.count(b);
    int start, len;
    bool first;  // whether a segment starts with the block
    blocks.at(b, n - 1, start, len, first);
    kn.load(block_rows(in.k, b, hk, start, len), in.k.st, 0, wd.k);
    if (!kShare) qn.load(block_rows(in.q, b, hk, start, len), in.q.st, 0, wd.k);
    on.load(block_rows(go, b, h, start, len), go.st, v0, wd.v);
    gn.load(in, prep, b, h, bh * s.T + start, start, len);
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
            for (int i = 0; i < ND; ++i) S[i] = f32x4{0, 0, 0, 0};
        } else {
            keep_state(keep.ds + (bh * slots + (behind < s.T ? behind / kC : slots - 1)) * s.K * kw, S);
        }
        kn.store(kt, kKPlane, KS);
        if (!kShare) qn.store(qt, kKPlane, KS);
        on.store(ot, kOPlane, VS);
        gn.store(gates);
#pragma unroll
        for (int i = 0; i < ND; ++i)
            store_planes(wide + (wc * 16 + ln) * KS + (wr * ND + i) * 16 + lg * 4, kSPlane, S[i]);
        __syncthreads();
        kn.load(block_rows(in.k, b, hk, prev, plen), in.k.st, 0, wd.k);
        if (kShare)
            qn.load(block_rows(in.q, b, hk, start, len), in.q.st, 0, wd.k);
        else
            qn.load(block_rows(in.q, b, hk, prev, plen), in.q.st, 0, wd.k);
        on.load(block_rows(go, b, h, prev, plen), go.st, v0, wd.v);
        gn.load(in, prep, b, h, bh * s.T + prev, prev, plen);

        f32x4 kd[NT], po[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) kd[i] = po[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KP / 32; ++k) {
            const Frag<3> sf = row_frag<3>(wide, kSPlane, KS, wc * 16, k * 32, lane);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma(kd[i], row_frag<NP>(kt, kKPlane, KS, (wr * NT + i) * 16, k * 32, lane), sf);
        }
        {
            const Frag<NP> o0 = col_frag<NP>(ot, kOPlane, VS, 0, wc * 16, lane);
            const Frag<NP> o1 = col_frag<NP>(ot, kOPlane, VS, 32, wc * 16, lane);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if (wr * NT + i < 2) mma(po[i], at[i][0], o0);
                mma(po[i], at[i][1], o1);
            }
        }
        load_cols(at, prep.att_t, prev, plen);
        f32x4 en[NT], be[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r0 = (wr * NT + i) * 16 + lg * 4;
            en[i] = *reinterpret_cast<const f32x4*>(gates + r0);
            be[i] = *reinterpret_cast<const f32x4*>(gates + 2 * kC + r0);
            const f32x4 le = *reinterpret_cast<const f32x4*>(gates + kC + r0);
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = fmaf(le[r], kd[i][r], in.scale * po[i][r]);
            store_planes(rt + (wc * 16 + ln) * kTS + r0, kTPlane, y);
        }
        const float end = gates[len - 1];
        __syncthreads();

        f32x4 x[NT];
        {
            const Frag<3> y0 = row_frag<3>(rt, kTPlane, kTS, wc * 16, 0, lane);
            const Frag<3> y1 = row_frag<3>(rt, kTPlane, kTS, wc * 16, 32, lane);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                x[i] = f32x4{0, 0, 0, 0};
                if (wr * NT + i < 2) mma(x[i], ti[i][0], y0);
                mma(x[i], ti[i][1], y1);
            }
        }
        load_cols(ti, prep.inv_t, prev, plen);
        keep_tokens(keep.r, start, len, x);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r0 = (wr * NT + i) * 16 + lg * 4;
            uint16_t* o = lt + (wc * 16 + ln) * kTS + r0;
            f32x4 l, e;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float dv = be[i][r] * x[i][r];
                l[r] = -en[i][r] * dv;
                e[r] = in.scale * en[i][r] * element<NP>(ot + (r0 + r) * VS + wc * 16 + ln, kOPlane);
                put1<DT>(gt, (r0 + r) * VS + wc * 16 + ln, dv);
            }
            store_planes(o, kTPlane, l);
            store_planes(o + 3 * kTPlane, kTPlane, e);
        }
        __syncthreads();
        store_rows<DT, W>(p.grad_v, gt, VS, s, b, h, start, len, v0, wd.out);

        {
            const Frag<3> l0 = row_frag<3>(lt, kTPlane, kTS, wc * 16, 0, lane);
            const Frag<3> l1 = row_frag<3>(lt, kTPlane, kTS, wc * 16, 32, lane);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] *= end;
                mma(S[i], col_frag<NP>(kt, kKPlane, KS, 0, (wr * ND + i) * 16, lane), l0);
                mma(S[i], col_frag<NP>(kt, kKPlane, KS, 32, (wr * ND + i) * 16, lane), l1);
            }
        }
        if (kShare) {
            __syncthreads();
            qn.store(qt, kKPlane, KS);
            __syncthreads();
        }
        {
            const Frag<3> e0 = row_frag<3>(et, kTPlane, kTS, wc * 16, 0, lane);
            const Frag<3> e1 = row_frag<3>(et, kTPlane, kTS, wc * 16, 32, lane);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                mma(S[i], col_frag<NP>(qt, kKPlane, KS, 0, (wr * ND + i) * 16, lane), e0);
                mma(S[i], col_frag<NP>(qt, kKPlane, KS, 32, (wr * ND + i) * 16, lane), e1);
            }
        }
        __syncthreads();
        start = prev, len = plen, cut = first, first = pfirst;
    }
    if (p.grad_h0)
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = (wr * ND + i) * 16 + lg * 4 + r;
                if (d < s.K && col < s.V) p.grad_h0[(bh * s.K + d) * s.V + col] = cut ? 0.0f : S[i][r];
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

// Contiguous rows of `bytes` that are whole aligned vectors.
bool whole(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)bytes) % 16 == 0; }

dim3 walk_grid(const DeltaShape& s, int groups) { return dim3((unsigned)((s.B * s.H + 7) / 8 * 8 * groups)); }

template <int DT, bool KEEP>
hipError_t walk(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaFwd& out,
                const Kept& keep, hipStream_t st) {
    const Widths wd{row_width(s.K, DT), row_width(s.V, DT), whole(out.out, s.V * Elem<DT>::bytes)};
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, CT = kMaxCT<DT, RT>;
        const int groups = (s.V + CT * 16 - 1) / (CT * 16);
        delta_walk<DT, RT, CT, KEEP><<<walk_grid(s, groups), kThreads, 0, st>>>(s, in, blocks, prep, out, keep, groups, wd);
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
    const Widths wd{row_width(s.K, DT), row_width(s.V, DT), whole(p.grad_v, s.V * Elem<DT>::bytes)};
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, CT = kMaxCT<DT, RT>;
        const int groups = (s.V + CT * 16 - 1) / (CT * 16);
        delta_walk_back<DT, RT, CT><<<walk_grid(s, groups), kThreads, 0, st>>>(s, in, blocks, prep, p, go, keep, groups, wd);
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
