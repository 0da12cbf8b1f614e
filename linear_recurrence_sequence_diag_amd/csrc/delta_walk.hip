// delta_walk.hip -- gated delta rule: the walk over a sequence's blocks that
// carries a head's state, forward and back.
//
// One wavefront carries 16 columns of one head's state [K, V] through all blocks of
// its batch row; the columns are independent.  With S of a block's start, a block's
// products follow one another,
//   K S -> X = (I + N)^-1 (V - enter K S) -> S' = end S + K^T (leave beta X),
// and O = scale (enter Q S + P beta X).  In the order of k described in
// delta_tile.hpp each result is the next product's operand where it stands, cut
// into bf16 planes in registers, so a wavefront waits for no other within a block.
// What does not depend on the columns (K, Q, rows of the inverse and of P) lies in
// LDS, shared by the up to eight wavefronts of a head that make up a workgroup; a
// block's is loaded into registers while the block before is at work.  Wavefronts
// beyond the columns only load.
//
// What bounds it is the length of a block's chain of products: bf16 [8, 2048], 20
// heads of 128 with resets, are 160 workgroups that take 17.3 thousand cycles a
// block, 288 us, 63 of them matrix instructions with two wavefronts a SIMD; LDS
// reads and the cutting into planes hardly overlap with these.  The kept walk of the
// backward pass takes 269 us (485 MB of states and x written), the walk back 365
// (579 MB).
#include "delta_tile.hpp"
#include "delta_ws.hpp"

#include <type_traits>

namespace lrscan {
namespace delta {

constexpr int kMaxWaves = 8;         // wavefronts with columns, at most; the launch says how many
constexpr int kTS = kC + 8;          // elements of an LDS row of 64
constexpr int kTPlane = kC * kTS;

// Workgroups of one head and part lie on one XCD, so its operands are read from
// memory once: the number of the two is the workgroup's number modulo 8.
__device__ __forceinline__ bool my_part(const DeltaShape& s, int groups, int parts, int64_t& bh, int& part, int& group) {
    const int r = (int)(blockIdx.x >> 3), x = scalar(r / groups) * 8 + (int)(blockIdx.x & 7);
    group = scalar(r % groups);
    part = scalar(x % parts);
    bh = scalar(x / parts);
    return bh < s.B * s.H;
}

// The blocks of a part: [first, end).
__device__ __forceinline__ void part_blocks(int n, int part, int parts, int& first, int& end) {
    first = scalar(part_start(n, part, parts));
    end = scalar(part_start(n, part + 1, parts));
}

// A block's gates, [3][kC] in LDS.
struct Gates {
    f32x4 x;
    __device__ __forceinline__ void load(const Prep& prep, int64_t t0, int len) {
        x = __builtin_bit_cast(f32x4, load16(buffer(prep.gates + t0, len * 16), threadIdx.x < kC ? threadIdx.x * 16 : kNowhere));
    }
    __device__ __forceinline__ void store(float* lds) const {
        const int i = threadIdx.x;
        if (i < kC) lds[i] = x[0], lds[kC + i] = x[1], lds[2 * kC + i] = x[2];
    }
};

// A tile of a block's kC rows and up to COLS columns (uniform `cols` of them, a
// multiple of 8), 8 columns a thread at a time; PLACED: columns stand in place().
template <int DT, int COLS, bool PLACED>
struct Tile {
    static constexpr int PER = kC * COLS / 8 / kWalkThreads;
    Raw8<DT> x[PER];
    __device__ __forceinline__ void load(Buffer rows, int64_t st, int c0, int cols, int n) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = i * kWalkThreads + threadIdx.x, q = o % (COLS / 8) * 8;
            x[i].load(rows, o / (COLS / 8) * (int)st, q < cols ? c0 + q : n, n);
        }
    }
    __device__ __forceinline__ void store(uint16_t* tile, int plane, int stride) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = i * kWalkThreads + threadIdx.x, q = o % (COLS / 8) * 8;
            uint16_t* row = tile + o / (COLS / 8) * stride;
            const auto f = x[i].frag();
            if constexpr (PLACED) {
#pragma unroll
                for (int p = 0; p < kPlanes<DT>; ++p) {
                    *reinterpret_cast<u32x2*>(row + p * plane + place(q)) = u32x2{f.p[p][0], f.p[p][1]};
                    *reinterpret_cast<u32x2*>(row + p * plane + place(q + 4)) = u32x2{f.p[p][2], f.p[p][3]};
                }
            } else {
                store_frag(row + q, plane, f);
            }
        }
    }
};

// V or dO of a block in LDS, [token][column], as they are stored: fp32 in one plane
// leaves room for eight wavefronts' columns beside K's 256 in three (fp32 [14, 513],
// 16 heads of 256: a forward call of 929 us, with four and V in three planes, took 693
// with them, and takes 670 now).
template <int DT, int COLS>
struct Values {
    static constexpr int kStride = DT == DT_F32 ? 2 * (COLS + 4) : COLS + 8, kSize = kC * kStride;
    static __device__ __forceinline__ void store(uint16_t* tile, const Tile<DT, COLS, false>& t) {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < t.PER; ++i) {
                const int o = i * kWalkThreads + threadIdx.x;
                f32x4* row = reinterpret_cast<f32x4*>(tile + o / (COLS / 8) * kStride + o % (COLS / 8) * 16);
                row[0] = t.x[i].a, row[1] = t.x[i].b;
            }
        } else {
            t.store(tile, 0, kStride);
        }
    }
    // a lane's four tokens of a column
    static __device__ __forceinline__ f32x4 four(const uint16_t* tile, int row0, int col0, int lane) {
        if constexpr (DT == DT_F32) {
            const float* at = reinterpret_cast<const float*>(tile) + (row0 + (lane >> 4) * 4) * (COLS + 4) + col0 + (lane & 15);
            return f32x4{at[0], at[COLS + 4], at[2 * (COLS + 4)], at[3 * (COLS + 4)]};
        } else {
            return read_values<1>(tile, 0, kStride, row0, col0, lane);
        }
    }
    // an operand with 32 tokens as k
    static __device__ __forceinline__ Frag<kPlanes<DT>> frag(const uint16_t* tile, int row0, int col0, int lane) {
        if constexpr (DT == DT_F32)
            return split8(four(tile, row0, col0, lane), four(tile, row0 + 16, col0, lane));
        else
            return rows_frag<1>(tile, 0, kStride, row0, col0, 4, lane);
    }
};

// A block's rows of kC in three planes.
struct Rows64 {
    u32x4 x[3];
    __device__ __forceinline__ void load(const uint16_t* p, int64_t t0, int len) {
        const Buffer rows = buffer(p + t0 * (3 * kC), len * (3 * kC * 2));
#pragma unroll
        for (int i = 0; i < 3; ++i) x[i] = load16(rows, (i * kWalkThreads + threadIdx.x) * 16);
    }
    __device__ __forceinline__ void store(uint16_t* tile) const {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int o = i * kWalkThreads + threadIdx.x, r = o / 24, q = o % 24;
            *reinterpret_cast<u32x4*>(tile + q / 8 * kTPlane + r * kTS + q % 8 * 8) = x[i];
        }
    }
};

// A lane's tokens of a column of a token scratch (rows of kw columns) and of a state
// scratch; what lies past rows or columns is left out.
__device__ __forceinline__ void keep_tokens(float* to, int kw, int len, int col, int lane, const f32x4 (&x)[4]) {
    const Buffer rows = buffer(to, (int64_t)len * kw * 4);
    const uint32_t at = anew(col < kw ? (uint32_t)(((lane >> 4) * 4 * kw + col) * 4) : kNowhere, reinterpret_cast<intptr_t>(to));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) store4(rows, at + (i * 16 + r) * kw * 4, x[i][r]);
}
template <int ND>
__device__ __forceinline__ void keep_state(float* to, int K, int kw, int col, int lane, const f32x4 (&x)[ND]) {
    const Buffer rows = buffer(to, (int64_t)K * kw * 4);
    const uint32_t at = anew(col < kw ? (uint32_t)(((lane >> 4) * 4 * kw + col) * 4) : kNowhere, reinterpret_cast<intptr_t>(to));
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) store4(rows, at + (i * 16 + r) * kw * 4, x[i][r]);
}
// The same of a state scratch, into accumulators.
template <int ND>
__device__ __forceinline__ void take_state(const float* from, int K, int kw, int col, int lane, f32x4 (&x)[ND]) {
    const Buffer rows = buffer(from, (int64_t)K * kw * 4);
    const uint32_t at = anew(col < kw ? (uint32_t)(((lane >> 4) * 4 * kw + col) * 4) : kNowhere, reinterpret_cast<intptr_t>(from));
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[i][r] = load4(rows, at + (i * 16 + r) * kw * 4);
}

// A column of a state [K, V] in or out of accumulators.
template <int ND, class F>
__device__ __forceinline__ void each_state(const DeltaShape& s, int64_t bh, int col, int lane, F f) {
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = i * 16 + (lane >> 4) * 4 + r;
            f(i, r, d < s.K && col < s.V, (bh * s.K + d) * s.V + col);
        }
}

// S = end S + K^T l (or Q^T l), l the tokens' two operands of 32.
template <int NP, int ND>
__device__ __forceinline__ void add_tokens(f32x4 (&S)[ND], const uint16_t* tile, int plane, int stride, const Frag<3>& l0,
                                           const Frag<3>& l1, int lane) {
#pragma unroll
    for (int i = 0; i < ND; i += 2) {
        f32x4 c[2] = {S[i], S[i + 1]};
        const Frag<NP> a[2] = {placed_rows_frag<NP>(tile, plane, stride, 0, i, lane),
                               placed_rows_frag<NP>(tile, plane, stride, 0, i + 1, lane)};
        const Frag<NP> b[2] = {placed_rows_frag<NP>(tile, plane, stride, 32, i, lane),
                               placed_rows_frag<NP>(tile, plane, stride, 32, i + 1, lane)};
        mma(c, a, l0);
        mma(c, b, l1);
        S[i] = c[0], S[i + 1] = c[1];
    }
}

// x += A y over a block's tokens, A's rows in LDS, y the tokens' two
// operands of 32; LOWER: rows reach the tokens up to their own, else from there on.
template <bool LOWER, int NB>
__device__ __forceinline__ void triangle(f32x4 (&x)[4], const uint16_t* rows, const Frag<NB>& y0, const Frag<NB>& y1,
                                         int lane) {
    f32x4 c[2] = {x[LOWER ? 2 : 0], x[LOWER ? 3 : 1]}, d[2] = {x[LOWER ? 0 : 2], x[LOWER ? 1 : 3]};
    const int full = LOWER ? 2 : 0, half = LOWER ? 0 : 2;  // tiles of rows with both operands, and with one
    const Frag<3> a[2] = {row_frag<3>(rows, kTPlane, kTS, full * 16, 0, lane),
                           row_frag<3>(rows, kTPlane, kTS, (full + 1) * 16, 0, lane)};
    const Frag<3> b[2] = {row_frag<3>(rows, kTPlane, kTS, full * 16, 32, lane),
                           row_frag<3>(rows, kTPlane, kTS, (full + 1) * 16, 32, lane)};
    const Frag<3> e[2] = {row_frag<3>(rows, kTPlane, kTS, half * 16, LOWER ? 0 : 32, lane),
                           row_frag<3>(rows, kTPlane, kTS, (half + 1) * 16, LOWER ? 0 : 32, lane)};
    mma(d, e, LOWER ? y0 : y1);
    mma(c, a, y0);
    mma(c, b, y1);
    x[full] = c[0], x[full + 1] = c[1], x[half] = d[0], x[half + 1] = d[1];
}

// A triangle's rows do not take all of the 32 tokens that a product spans: the others'
// weights are zeros, which leave a value out unless it is not finite.  So from a
// column's first such token on (of the triangle that reaches back, up to its last
// one) an operand is zeros, and the rows that do take it are made NaN afterwards.
// What rounds to an infinity in bf16 counts as one.  Looking for such tokens is 1 to
// 3% of a call (bf16 [8, 2048], 20 heads of 128: 3 us of 370, reverse 17 of 1320),
// which without the branches marked as rare is 12%: spills.
constexpr float kOver = 0x1.ffp127f;
template <bool LOWER>
__device__ __forceinline__ int mute(f32x4 (&y)[4], int lane) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) most = __builtin_elementwise_maximum(most, fabsf(y[i][r]));  // NaN where there is one
    int at = LOWER ? kC : -1;
    if (__builtin_expect(__any(!(most < kOver)), 0)) {
        auto each = [&](auto f) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) f(i * 16 + (lane >> 4) * 4 + r, i, r);
        };
        each([&](int t, int i, int r) {
            if (!(fabsf(y[i][r]) < kOver)) at = LOWER ? min(at, t) : max(at, t);
        });
#pragma unroll
        for (int m = 16; m < 64; m *= 2) {
            const int other = __shfl_xor(at, m);
            at = LOWER ? min(at, other) : max(at, other);
        }
        each([&](int t, int i, int r) {
            if (LOWER ? t >= at : t <= at) y[i][r] = 0.0f;
        });
    }
    return at;
}
template <bool LOWER>
__device__ __forceinline__ void spoil(f32x4 (&x)[4], int at, int lane) {
    if (__builtin_expect(!__any(LOWER ? at < kC : at >= 0), 1)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = i * 16 + (lane >> 4) * 4 + r;
            if (LOWER ? t >= at : t <= at) x[i][r] = __builtin_nanf("");
        }
}

// Elements of the operands' rows of K and of V.
struct Widths {
    int k, v;
};

// What a walk leaves: outputs and the last state; x and the states that enter
// blocks; or, of a part, the map from the state that enters it to the one that
// leaves: columns of V from zero, then K columns of the identity with values of 0.
enum Leaves { kOutputs, kKept, kSpan };

template <int DT, int RT, int LEAVES>
__global__ void __launch_bounds__(kWalkThreads, 2)
delta_walk(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaFwd p, Kept keep, Parts parts, int groups, int waves, Widths wd) {
    constexpr bool KEEP = LEAVES != kOutputs;
    constexpr int NP = kPlanes<DT>;
    constexpr int ND = 4 * RT, KP = 64 * RT, KS = KP + 8, kKPlane = kC * KS;
    using Columns = Values<DT, 16 * kMaxWaves>;
    // fp32 tiles take three planes each: of more than 64 rows Q lies where K will, the
    // inverse where P will (of 64 with room for all, fp32 [4, 1023, 16 heads of 64]
    // reverse 241 us a call for 248)
    constexpr bool kShare = DT == DT_F32 && RT > 1;
    __shared__ __attribute__((aligned(16))) uint16_t kt[NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t qt_[KEEP || kShare ? 8 : NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t it[3 * kTPlane];
    __shared__ __attribute__((aligned(16))) uint16_t at_[KEEP || kShare ? 8 : 3 * kTPlane];
    __shared__ __attribute__((aligned(16))) uint16_t vt[Columns::kSize];  // V [token][column]
    __shared__ __attribute__((aligned(16))) float gates[3 * kC];
    uint16_t *const qt = kShare ? kt : qt_, *const at = kShare ? it : at_;

    int64_t bh;
    int group, part;
    // of the last part nothing needs the map, and of the first only where the initial state leads
    if (!my_part(s, groups, LEAVES == kSpan ? parts.n - 1 : parts.n, bh, part, group)) return;
    const int64_t b = scalar((int)bh / s.H);
    const int h = scalar((int)bh % s.H), hk = scalar(h / (s.H / s.HK));
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int v0 = group * waves * 16, col = v0 + w * 16 + ln, kw = kept_width(s.V);
    const bool works = w < waves;
    const int one = LEAVES == kSpan ? col - (s.V + 15) / 16 * 16 : -1;  // the column of the identity

    f32x4 S[ND];
    if (LEAVES != kSpan && part > 0)
        take_state<ND>(parts.enter + (bh * parts.n + part) * s.K * kw, s.K, kw, works ? col : kw, lane, S);
    else
        each_state<ND>(s, bh, col, lane, [&](int i, int r, bool ok, int64_t at) {
            S[i][r] = works && part == 0 && in.h0 && ok ? in.h0[at] : i * 16 + lg * 4 + r == one ? 1.0f : 0.0f;
        });

    Tile<DT, KP, true> kn, qn;
    Tile<DT, 16 * kMaxWaves, false> vn;
    Rows64 tn, an;
    Gates gn;
    // what shares a place follows later, so that not all of a block is in registers
    // (fp32 forward calls: [8, 1024], 16 heads of 128, 224 us for 234; [14, 513], 16
    // heads of 192, 384 for 436, of 256 668 for 674)
    constexpr bool kLater = !KEEP && kShare;
    auto load_later = [&](int start, int len) {
        kn.load(block_rows(in.k, b, hk, start, len), in.k.st, 0, KP, wd.k);
        if (!KEEP) an.load(prep.att, bh * s.T + start, len);
    };
    auto load = [&](int start, int len) {
        gn.load(prep, bh * s.T + start, len);
        if (!KEEP) qn.load(block_rows(in.q, b, hk, start, len), in.q.st, 0, KP, wd.k);
        vn.load(block_rows(in.v, b, h, start, len), in.v.st, v0, waves * 16, wd.v);
        tn.load(prep.inv, bh * s.T + start, len);
        if (!kLater) load_later(start, len);
    };
    int from, n;
    part_blocks(blocks.count(b), part, parts.n, from, n);
    int start, len;
    bool cut;
    blocks.at(b, from, start, len, cut);
    load(start, len);
    for (int c = from; c < n; ++c) {
        // the next block; past the last one, one without tokens
        int next = s.T, nlen = 0;
        bool ncut = false;
        if (c + 1 < n) blocks.at(b, c + 1, next, nlen, ncut);
        gn.store(gates);
        if (!KEEP) qn.store(qt, kKPlane, KS);
        if (KEEP || !kShare) kn.store(kt, kKPlane, KS);
        Columns::store(vt, vn);
        tn.store(it);
        if (!KEEP && !kShare) an.store(at);
        __syncthreads();
        if (kLater)
            load_later(start, len);
        else
            load(next, nlen);

        f32x4 qs[4], ks[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qs[i] = ks[i] = f32x4{0, 0, 0, 0};
        if (works) {
            if (cut) {
#pragma unroll
                for (int i = 0; i < ND; ++i) S[i] = f32x4{0, 0, 0, 0};
            } else if (LEAVES == kKept) {
                keep_state<ND>(keep.s + (bh * state_slots(s.T) + entering_slot(start)) * s.K * kw, s.K, kw, col, lane, S);
            }
        }
        // x += A S for rows A in LDS
        auto times_state = [&](f32x4 (&x)[4], const uint16_t* tile, const auto& sf, int g) {
            Frag<NP> a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = row_frag<NP>(tile, kKPlane, KS, i * 16, g * 32, lane);
            mma(x, a, sf);
        };
        if (works) {
#pragma unroll
            for (int g = 0; g < KP / 32; ++g) {
                const Frag<3> sf = split8(S[2 * g], S[2 * g + 1]);
                if (!KEEP) times_state(qs, qt, sf, g);
                if (KEEP || !kShare) times_state(ks, kt, sf, g);
            }
        }
        if (!KEEP && kShare) {
            __syncthreads();  // Q is read
            kn.store(kt, kKPlane, KS);
            __syncthreads();
            load(next, nlen);
            if (works)
#pragma unroll
                for (int g = 0; g < KP / 32; ++g) {
                    times_state(ks, kt, split8(S[2 * g], S[2 * g + 1]), g);
                }
        }
        f32x4 en[4];
        Frag<3> l0, l1, u0, u1;
        float end = 0.0f;
        int bad = kC;  // the column's first token whose value is not finite
        if (works) {
            end = gates[len - 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                en[i] = *reinterpret_cast<const f32x4*>(gates + i * 16 + lg * 4);
                const f32x4 v = Columns::four(vt, i * 16, w * 16, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) ks[i][r] = fmaf(-en[i][r], ks[i][r], v[r]);
            }
            f32x4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f32x4{0, 0, 0, 0};
            bad = mute<true>(ks, lane);
            triangle<true>(x, it, split8(ks[0], ks[1]), split8(ks[2], ks[3]), lane);
            spoil<true>(x, bad, lane);
            if (LEAVES == kKept) keep_tokens(keep.x + (bh * s.T + start) * kw, kw, len, col, lane, x);
            f32x4 l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 le = *reinterpret_cast<const f32x4*>(gates + kC + i * 16 + lg * 4);
                const f32x4 be = *reinterpret_cast<const f32x4*>(gates + 2 * kC + i * 16 + lg * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[i][r] *= be[r];
                    l[i][r] = le[r] * x[i][r];
                }
            }
            if (!KEEP) bad = mute<true>(x, lane);
            u0 = split8(x[0], x[1]), u1 = split8(x[2], x[3]);
            l0 = split8(l[0], l[1]), l1 = split8(l[2], l[3]);
        }
        if (!KEEP && kShare) {
            __syncthreads();  // the inverse is read
            an.store(at);
            __syncthreads();
        }
        if (works) {
            if (!KEEP && p.out) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) qs[i][r] *= en[i][r];
                triangle<true>(qs, at, u0, u1, lane);
                spoil<true>(qs, bad, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) qs[i][r] *= in.scale;
                store_tokens<DT, 4>(p.out, b * s.T + start, len, s.H, h, s.V, 0, col, lane, qs);
            }
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] *= end;
            add_tokens<NP>(S, kt, kKPlane, KS, l0, l1, lane);
        }
        __syncthreads();  // all of the block is read
        start = next, len = nlen, cut = ncut;
    }
    if (LEAVES == kSpan && works) {
        if (one < 0) {
            keep_state<ND>(parts.enter + (bh * parts.n + part + 1) * s.K * kw, s.K, kw, col, lane, S);
        } else if (part > 0) {
            const int64_t at = (bh * parts.n + part) * s.K * kept_width(s.K);
            keep_state<ND>(parts.map + at, s.K, kept_width(s.K), one, lane, S);
            if (parts.map_t) {
                const Buffer rows = buffer(parts.map_t + at, (int64_t)s.K * kept_width(s.K) * 4);
#pragma unroll
                for (int i = 0; i < ND; ++i) {
                    const int d = i * 16 + lg * 4;
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[i]), rows,
                                                           d < kept_width(s.K) ? (one * kept_width(s.K) + d) * 4 : kNowhere, 0, 0);
                }
            }
        }
    }
    if (!KEEP && p.last && works && part + 1 == parts.n)
        each_state<ND>(s, bh, col, lane, [&](int i, int r, bool ok, int64_t at) {
            if (ok) p.last[at] = S[i][r];
        });
}

// The walk back.  With P the outputs' weights, dS the gradient of the state
// that leaves a block and everything scaled as above,
//   dU = scale P^T dO + leave K dS,  R = (I + diag(beta) M)^-T dU  (the gradient
//   of beta (V - enter K S)),  dV = beta R,
//   dS' = end dS + Q^T (scale enter dO) - K^T (beta enter R).
// SPAN: of a part only the gradient that reaches the state entering it, from
// nothing behind it (of the last part, from grad_last).
template <int DT, int RT, bool SPAN>
__global__ void __launch_bounds__(kWalkThreads, 2)
delta_walk_back(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaBwd p, HeadRows go, Kept keep, Parts parts,
                int groups, int waves, Widths wd) {
    constexpr int NP = kPlanes<DT>;
    constexpr int ND = 4 * RT, KP = 64 * RT, KS = KP + 8, kKPlane = kC * KS;
    using Columns = Values<DT, 16 * kMaxWaves>;
    // fp32 of more than 64 rows: Q follows K in one place, the inverse P in another
    constexpr bool kShare = DT == DT_F32 && RT > 1;
    __shared__ __attribute__((aligned(16))) uint16_t kt[NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t qt_[kShare ? 8 : NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t at[3 * kTPlane];
    __shared__ __attribute__((aligned(16))) uint16_t it_[kShare ? 8 : 3 * kTPlane];
    __shared__ __attribute__((aligned(16))) uint16_t ot[Columns::kSize];  // dO [token][column]
    __shared__ __attribute__((aligned(16))) float gates[3 * kC];
    uint16_t *const qt = kShare ? kt : qt_, *const it = kShare ? at : it_;

    int64_t bh;
    int group, part;
    if (!my_part(s, groups, SPAN ? parts.n - 1 : parts.n, bh, part, group)) return;
    if (SPAN) ++part;  // nothing needs it of the first
    const int64_t b = scalar((int)bh / s.H);
    const int h = scalar((int)bh % s.H), hk = scalar(h / (s.H / s.HK));
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int v0 = group * waves * 16, col = v0 + w * 16 + ln, kw = kept_width(s.V);
    const bool works = w < waves;
    const int64_t slots = state_slots(s.T);

    f32x4 S[ND];
    if (!SPAN && part + 1 < parts.n)
        take_state<ND>(parts.leave + (bh * parts.n + part) * s.K * kw, s.K, kw, works ? col : kw, lane, S);
    else
        each_state<ND>(s, bh, col, lane, [&](int i, int r, bool ok, int64_t at) {
            S[i][r] = works && part + 1 == parts.n && p.grad_last && ok ? p.grad_last[at] : 0.0f;
        });

    Tile<DT, KP, true> kn, qn;
    Tile<DT, 16 * kMaxWaves, false> on;
    Rows64 tn, an;
    Gates gn;
    // what shares a place follows later (fp32 [14, 513], 16 heads of 192, reverse: 1165 us
    // for 1210; of 256 1712 for 1744)
    auto load_later = [&](int start, int len) {
        tn.load(prep.inv_t, bh * s.T + start, len);
        qn.load(block_rows(in.q, b, hk, start, len), in.q.st, 0, KP, wd.k);
    };
    auto load = [&](int start, int len) {
        gn.load(prep, bh * s.T + start, len);
        kn.load(block_rows(in.k, b, hk, start, len), in.k.st, 0, KP, wd.k);
        on.load(block_rows(go, b, h, start, len), go.st, v0, waves * 16, wd.v);
        an.load(prep.att_t, bh * s.T + start, len);
        if (!kShare) load_later(start, len);
    };
    const int count = blocks.count(b);
    int to, n;
    part_blocks(count, part, parts.n, to, n);
    int start, len;
    bool first;  // whether a segment starts with the block
    blocks.at(b, n - 1, start, len, first);
    load(start, len);
    // what leaves a block enters the one behind it, unless a segment starts there: then
    // it is kept nowhere, as its place may be that of a block in another part
    bool cut = blocks.cut_behind(b, n - 1, count);
    for (int c = n - 1; c >= to; --c) {
        const int behind = start + len;
        int prev = 0, plen = 0;
        bool pfirst = false;
        if (c > to) blocks.at(b, c - 1, prev, plen, pfirst);
        gn.store(gates);
        kn.store(kt, kKPlane, KS);
        Columns::store(ot, on);
        an.store(at);
        if (!kShare) {
            tn.store(it);
            qn.store(qt, kKPlane, KS);
        }
        __syncthreads();
        if (kShare)
            load_later(start, len);
        else
            load(prev, plen);

        f32x4 x[4], po[4], en[4];
        Frag<NP> o0, o1;
        float end = 0.0f;
        if (works) {
            if (cut) {
#pragma unroll
                for (int i = 0; i < ND; ++i) S[i] = f32x4{0, 0, 0, 0};
            } else if (!SPAN) {
                keep_state<ND>(keep.ds + (bh * slots + leaving_slot(s.T, behind)) * s.K * kw, s.K, kw, col, lane, S);
            }
            end = gates[len - 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = po[i] = f32x4{0, 0, 0, 0};
                en[i] = *reinterpret_cast<const f32x4*>(gates + i * 16 + lg * 4);
            }
            o0 = Columns::frag(ot, 0, w * 16, lane);
            o1 = Columns::frag(ot, 32, w * 16, lane);
            triangle<false>(po, at, o0, o1, lane);
            // a gradient that is not finite stands in every row of the first tile
            if (__builtin_expect(__any(!(fabsf(po[0][0]) < INFINITY)), 0)) {
                f32x4 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i] = Columns::four(ot, i * 16, w * 16, lane);
                    po[i] = f32x4{0, 0, 0, 0};
                }
                const int bad = mute<false>(o, lane);
                triangle<false>(po, at, split8(o[0], o[1]), split8(o[2], o[3]), lane);
                spoil<false>(po, bad, lane);
            }
#pragma unroll
            for (int g = 0; g < KP / 32; ++g) {
                const Frag<3> sf = split8(S[2 * g], S[2 * g + 1]);
                Frag<NP> a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = row_frag<NP>(kt, kKPlane, KS, i * 16, g * 32, lane);
                mma(x, a, sf);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 le = *reinterpret_cast<const f32x4*>(gates + kC + i * 16 + lg * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) po[i][r] = fmaf(le[r], x[i][r], in.scale * po[i][r]);
            }
        }
        if (kShare) {
            __syncthreads();  // the weights are read
            tn.store(it);
            __syncthreads();
        }
        if (works) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f32x4{0, 0, 0, 0};
            const int bad = mute<false>(po, lane);
            triangle<false>(x, it, split8(po[0], po[1]), split8(po[2], po[3]), lane);
            spoil<false>(x, bad, lane);
            if (!SPAN) keep_tokens(keep.r + (bh * s.T + start) * kw, kw, len, col, lane, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 be = *reinterpret_cast<const f32x4*>(gates + 2 * kC + i * 16 + lg * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[i][r] *= be[r];
                    po[i][r] = -en[i][r] * x[i][r];
                }
            }
            if (!SPAN) store_tokens<DT, 4>(p.grad_v, b * s.T + start, len, s.H, h, s.V, 0, col, lane, x);
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] *= end;
            add_tokens<NP>(S, kt, kKPlane, KS, split8(po[0], po[1]), split8(po[2], po[3]), lane);
        }
        if (kShare) {
            __syncthreads();  // K is read
            qn.store(qt, kKPlane, KS);
            __syncthreads();
            load(prev, plen);
        }
        if (works) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 o = Columns::four(ot, i * 16, w * 16, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[i][r] = in.scale * en[i][r] * o[r];
            }
            add_tokens<NP>(S, qt, kKPlane, KS, split8(x[0], x[1]), split8(x[2], x[3]), lane);
        }
        __syncthreads();  // all of the block is read
        start = prev, len = plen, cut = first, first = pfirst;
    }
    if (SPAN && works) {
        if (cut)
#pragma unroll
            for (int i = 0; i < ND; ++i) S[i] = f32x4{0, 0, 0, 0};
        keep_state<ND>(parts.leave + (bh * parts.n + part - 1) * s.K * kw, s.K, kw, col, lane, S);
    }
    if (!SPAN && p.grad_h0 && works && part == 0) {
        // without an initial state the blocks leave its decay out
        const float decay = in.h0 ? 1.0f : expf(*reinterpret_cast<const float*>(in.g.row(b, 0, h)));
        each_state<ND>(s, bh, col, lane, [&](int i, int r, bool ok, int64_t at) {
            if (ok) p.grad_h0[at] = cut ? 0.0f : decay * S[i][r];
        });
    }
}

// ---- parts of a long sequence ----
//
// A sequence over few heads is walked in parts at the same time: first every part's
// map S -> A S + B is formed, then the states between parts, one after the other,
// then each part is walked from its own.  The gradients' maps are the transposed
// ones.  Here the states between: x[p + 1] += A_p x[p], forward, for p from 1 on,
// or x[p - 1] += A_p^T x[p] back, for p from parts - 2 on; a workgroup has 16
// columns of a head, its wavefronts tiles of 16 rows.  A part that a segment starts
// in passes nothing on, which no product says: what it is handed, and its map past
// the start, may be infinite.
// A step waits for the one before it, so its map is loaded while that one is at
// work, where the registers hold both (bf16, 8 heads of 128: 2.5 us a step, 3.1
// when loaded within it; what bounds it is a compute unit's 64 KB of map a step).
constexpr int kJoinS = kDeltaMaxK + 8;

template <bool BACK, int RT>
__global__ void __launch_bounds__(kWalkThreads, 2) delta_join(DeltaShape s, Blocks blocks, Parts parts, int tiles) {
    constexpr int NT = RT > 2 ? 2 : 1, NK = 2 * RT;  // a wavefront's tiles, and their operands of 32
    constexpr bool kAhead = RT <= 2;                 // registers hold two steps' maps
    __shared__ __attribute__((aligned(16))) uint16_t xs[2][3 * 16 * kJoinS];
    __shared__ bool barred[kComputeUnits];  // parts that a segment starts in
    static_assert(kComputeUnits <= kWalkThreads, "a thread for each part");
    // workgroups of a head lie on one XCD and read its maps once
    const int r8 = (int)(blockIdx.x >> 3);
    const int64_t bh = scalar(r8 / tiles * 8 + (int)(blockIdx.x & 7));
    if (bh >= s.B * s.H) return;
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int col = r8 % tiles * 16 + ln, kw = kept_width(s.V), ka = kept_width(s.K);
    const int64_t state = (int64_t)s.K * kw;
    float* const x = (BACK ? parts.leave : parts.enter) + bh * parts.n * state;
    const float* const map = (BACK ? parts.map_t : parts.map) + bh * parts.n * s.K * ka;
    auto tile_at = [&](int i) { return col < kw ? (uint32_t)(((i * 16 + lg * 4) * kw + col) * 4) : kNowhere; };
    const int first = BACK ? parts.n - 2 : 1, by = BACK ? -1 : 1, steps = parts.n - 2;
    if (threadIdx.x < parts.n) {
        const int64_t b = bh / s.H;
        const int n = blocks.count(b), part = (int)threadIdx.x, end = part_start(n, part + 1, parts.n);
        bool any = false;
        for (int c = part_start(n, part, parts.n); c < end && !any; ++c) {
            int start, len;
            blocks.at(b, c, start, len, any);
        }
        barred[threadIdx.x] = any;
    }
    for (int i = w; i < kDeltaMaxK / 16; i += 8) {  // past the rows: zeros
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = load4(buffer(x + first * state, state * 4), tile_at(i) + r * kw * 4);
        store_planes(xs[0] + ln * kJoinS + i * 16 + lg * 4, 16 * kJoinS, v);
        store_planes(xs[1] + ln * kJoinS + i * 16 + lg * 4, 16 * kJoinS, f32x4{0, 0, 0, 0});
    }
    struct Operands {
        Raw8<DT_F32> a[NT][NK];
        f32x4 own[NT];
    } x0, x1;
    auto state_of = [&](int step) {  // nothing past the last step
        return buffer(x + (first + by * (step + 1)) * state, step < steps ? state * 4 : 0);
    };
    auto load = [&](Operands& o, int step) {
        const Buffer rows = buffer(map + (int64_t)(first + by * step) * s.K * ka, step < steps ? (int64_t)s.K * ka * 4 : 0);
        const Buffer own = state_of(step);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < NK; ++j) o.a[t][j].load(rows, ((w + 8 * t) * 16 + ln) * ka * 4, j * 32 + lg * 8, ka);
#pragma unroll
            for (int r = 0; r < 4; ++r) o.own[t][r] = load4(own, tile_at(w + 8 * t) + r * kw * 4);
        }
    };
    auto join = [&](int step, Operands& o, Operands& next) {
        const Buffer out = state_of(step);
        const bool through = !barred[first + by * step];
        const uint16_t* now = xs[step & 1];
        uint16_t* then = xs[1 - (step & 1)];
        if (kAhead) {
            load(next, step + 1);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int j = 0; j < NK; ++j)
                mma(c[j & 1], o.a[t][j].frag(), row_frag<3>(now, 16 * kJoinS, kJoinS, 0, j * 32, lane));
            const int i = w + 8 * t;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                c[0][r] = o.own[t][r] + (through ? c[0][r] + c[1][r] : 0.0f);
                store4(out, tile_at(i) + r * kw * 4, c[0][r]);
            }
            store_planes(then + ln * kJoinS + i * 16 + lg * 4, 16 * kJoinS, c[0]);
        }
        if (!kAhead) load(o, step + 1);
        __syncthreads();
    };
    load(x0, 0);
    __syncthreads();
    for (int step = 0; step < steps; step += kAhead ? 2 : 1) {
        join(step, x0, x1);
        if (kAhead && step + 1 < steps) join(step + 1, x1, x0);
    }
}

template <class F>
hipError_t by_rows(const DeltaShape& s, F f) {
    switch ((s.K + 63) / 64) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        default: return f(std::integral_constant<int, 4>{});
    }
}

hipError_t run_join(const DeltaShape& s, const Blocks& blocks, const Parts& parts, bool back, hipStream_t st) {
    if (parts.n < 3) return hipSuccess;
    const int tiles = (s.V + 15) / 16;
    const dim3 grid((unsigned)((s.B * s.H + 7) / 8 * 8 * tiles));
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value;
        if (back)
            delta_join<true, RT><<<grid, kWalkThreads, 0, st>>>(s, blocks, parts, tiles);
        else
            delta_join<false, RT><<<grid, kWalkThreads, 0, st>>>(s, blocks, parts, tiles);
        return hipGetLastError();
    });
}

struct Spread {
    int waves, groups;
    dim3 grid;
};

// Columns are spread evenly over the workgroups of a head, on more of them than
// need be where that leaves compute units idle: a block then takes less time
// (us of a call without parts, 8, 4, 2 and 1 wavefronts a workgroup: bf16 [1, 32768,
// 8 heads of 128] 3438, 2252, 2218, 2217; fp32 [4, 1023, 16 heads of 64] reverse 276,
// 276, 270, 269; but of 160 heads bf16 [8, 2048] 336, 394, 529, 809).
Spread spread(const DeltaShape& s, int tiles, int parts, int most) {
    const int64_t heads = s.B * s.H * parts, spare = kComputeUnits / heads;
    int groups = (tiles + most - 1) / most;
    if (spare > groups) groups = spare < tiles ? (int)spare : tiles;
    const int waves = (tiles + groups - 1) / groups;
    groups = (tiles + waves - 1) / waves;
    return Spread{waves, groups, dim3((unsigned)((heads + 7) / 8 * 8 * groups))};
}

template <int DT, int LEAVES>
hipError_t walk(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaFwd& out,
                const Kept& keep, const Parts& parts, hipStream_t st) {
    const Widths wd{row_width(s.K, DT), row_width(s.V, DT)};
    const int tiles = (s.V + 15) / 16 + (LEAVES == kSpan ? (s.K + 15) / 16 : 0);
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value;
        const Spread x = spread(s, tiles, LEAVES == kSpan ? parts.n - 1 : parts.n, kMaxWaves);
        delta_walk<DT, RT, LEAVES>
            <<<x.grid, kWalkThreads, 0, st>>>(s, in, blocks, prep, out, keep, parts, x.groups, x.waves, wd);
        return hipGetLastError();
    });
}

hipError_t run_walk(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                    const DeltaFwd& out, const Kept* keep, const Parts& parts, hipStream_t st) {
    if (parts.n > 1) {
        const hipError_t e = s.dtype == DT_F32 ? walk<DT_F32, kSpan>(s, in, blocks, prep, out, Kept{}, parts, st)
                                               : walk<DT_BF16, kSpan>(s, in, blocks, prep, out, Kept{}, parts, st);
        if (e != hipSuccess) return e;
        const hipError_t f = run_join(s, blocks, parts, false, st);
        if (f != hipSuccess) return f;
    }
    if (s.dtype == DT_F32)
        return keep ? walk<DT_F32, kKept>(s, in, blocks, prep, out, *keep, parts, st)
                    : walk<DT_F32, kOutputs>(s, in, blocks, prep, out, Kept{}, parts, st);
    return keep ? walk<DT_BF16, kKept>(s, in, blocks, prep, out, *keep, parts, st)
                : walk<DT_BF16, kOutputs>(s, in, blocks, prep, out, Kept{}, parts, st);
}

template <int DT, bool SPAN>
hipError_t walk_back(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaBwd& p,
                     const HeadRows& go, const Kept& keep, const Parts& parts, hipStream_t st) {
    const Widths wd{row_width(s.K, DT), row_width(s.V, DT)};
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value;
        const Spread x = spread(s, (s.V + 15) / 16, SPAN ? parts.n - 1 : parts.n, kMaxWaves);
        delta_walk_back<DT, RT, SPAN>
            <<<x.grid, kWalkThreads, 0, st>>>(s, in, blocks, prep, p, go, keep, parts, x.groups, x.waves, wd);
        return hipGetLastError();
    });
}

hipError_t run_walk_back(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                         const DeltaBwd& p, const HeadRows& go, const Kept& keep, const Parts& parts, hipStream_t st) {
    const bool wide = s.dtype == DT_F32;
    if (parts.n > 1) {
        hipError_t e = wide ? walk_back<DT_F32, true>(s, in, blocks, prep, p, go, keep, parts, st)
                            : walk_back<DT_BF16, true>(s, in, blocks, prep, p, go, keep, parts, st);
        if (e == hipSuccess) e = run_join(s, blocks, parts, true, st);
        if (e != hipSuccess) return e;
    }
    return wide ? walk_back<DT_F32, false>(s, in, blocks, prep, p, go, keep, parts, st)
                : walk_back<DT_BF16, false>(s, in, blocks, prep, p, go, keep, parts, st);
}

}  // namespace delta
}  // namespace lrscan
