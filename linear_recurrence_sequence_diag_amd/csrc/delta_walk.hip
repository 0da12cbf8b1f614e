// delta_walk.hip -- gated delta rule: the walk over a sequence's blocks that
// carries a head's state, forward and back.
//
// One workgroup carries CT * 16 columns of one head's state [K, V] through all
// blocks of its batch row; the columns are independent.  Its four wavefronts
// hold the state's rows in accumulators (16 RT rows each) and take 16 tokens of
// a block each.  A block's products follow one another,
//   K S -> X = (I + N)^-1 (V - enter K S) -> S' = end S + K^T (leave beta X),
// and each result becomes the next one's operand through LDS, cut into bf16
// planes there.  Q S and the outputs' product with U fill in beside them.
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

template <int DT, int RT, int CT, bool KEEP>
__global__ void __launch_bounds__(kThreads) delta_walk(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaFwd p,
                                                       Kept keep, int groups, bool vec) {
    constexpr int NP = kPlanes<DT>;
    constexpr int KP = 64 * RT;      // rows of the state, padded
    constexpr int KS = KP + 8;       // elements of an LDS row of K
    constexpr int W = CT * 16;       // columns
    constexpr int kKPlane = kC * KS, kSPlane = W * KS, kTPlane = W * kTS;
    constexpr int kWide = 3 * (kSPlane > 2 * kTPlane ? kSPlane : 2 * kTPlane);
    __shared__ __attribute__((aligned(16))) uint16_t kt[NP * kKPlane];  // K of the block [token][row]
    __shared__ __attribute__((aligned(16))) uint16_t wide[kWide];       // the state, then u and leave u
    __shared__ __attribute__((aligned(16))) uint16_t rt[3 * kTPlane];   // right sides of the triangular system
    __shared__ __attribute__((aligned(16))) float enter[kC], leave[kC], beta[kC];
    uint16_t *const ut = wide, *const lt = wide + 3 * kTPlane;

    int64_t bh;
    int group;
    if (!my_head(s, groups, bh, group)) return;
    const int64_t b = bh / s.H;
    const int h = (int)(bh % s.H), hk = h / (s.H / s.HK);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, ln = lane & 15, lg = lane >> 4;
    const int v0 = group * W;

    f32x4 S[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = (w * RT + i) * 16 + lg * 4 + r, col = v0 + j * 16 + ln;
                S[i][j][r] = in.h0 && d < s.K && col < s.V ? in.h0[(bh * s.K + d) * s.V + col] : 0.0f;
            }

    const int n = blocks.count(b);
    for (int c = 0; c < n; ++c) {
        int start, len;
        blocks.at(b, c, start, len);
        const int row = w * 16 + ln;
        if (in.reset && in.reset[b * s.T + start]) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j) S[i][j] = f32x4{0, 0, 0, 0};
        } else if (KEEP) {
            float* to = keep.s + (bh * state_slots(s.T) + start / kC) * s.K * s.V;
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int d = (w * RT + i) * 16 + lg * 4 + r, col = v0 + j * 16 + ln;
                        if (d < s.K && col < s.V) to[(int64_t)d * s.V + col] = S[i][j][r];
                    }
        }
        // rows of the inverse and of the outputs' weights, for the products below
        Raw8<DT_F32> ti[2], at[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int64_t o = (bh * s.T + start + row) * kC + ks * 32 + lg * 8;
            const bool ok = row < len && (ks == 0 || w >= 2);
            load8(ti[ks], reinterpret_cast<const char*>(prep.inv + o), ok, 0, 8, true);
            if (!KEEP) load8(at[ks], reinterpret_cast<const char*>(prep.att + o), ok, 0, 8, true);
        }
        // K into LDS
        for (int i = threadIdx.x; i < kC * KP / 8; i += kThreads) {
            const int r = i / (KP / 8), q = i % (KP / 8) * 8;
            Raw8<DT> x;
            load8(x, in.k.row(b, start + r, hk), r < len, q, s.K, vec);
            store_frag(kt + r * KS + q, kKPlane, x.frag());
        }
        if (threadIdx.x < kC) {
            const bool ok = threadIdx.x < len;
            const int64_t o = bh * s.T + start + threadIdx.x;
            enter[threadIdx.x] = ok ? prep.enter[o] : 0.0f;
            leave[threadIdx.x] = ok ? prep.leave[o] : 0.0f;
            beta[threadIdx.x] = ok ? *reinterpret_cast<const float*>(in.beta.row(b, start + threadIdx.x, h)) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j)
                store_planes(wide + (j * 16 + ln) * KS + (w * RT + i) * 16 + lg * 4, kSPlane, S[i][j]);
        __syncthreads();

        f32x4 ks_[CT], qs[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) ks_[j] = qs[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k0 = 0; k0 < KP; k0 += 32) {
            const Frag<NP> kf = row_frag<NP>(kt, kKPlane, KS, w * 16, k0, lane);
            Frag<NP> qf;
            if (!KEEP) {
                Raw8<DT> q;
                load8(q, in.q.row(b, start + row, hk), row < len, k0 + lg * 8, s.K, vec);
                qf = q.frag();
            }
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const Frag<3> sf = row_frag<3>(wide, kSPlane, KS, j * 16, k0, lane);
                mma(ks_[j], kf, sf);
                if (!KEEP) mma(qs[j], qf, sf);
            }
        }
        const f32x4 en = *reinterpret_cast<const f32x4*>(enter + w * 16 + lg * 4);
        const f32x4 le = *reinterpret_cast<const f32x4*>(leave + w * 16 + lg * 4);
        const f32x4 be = *reinterpret_cast<const f32x4*>(beta + w * 16 + lg * 4);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = w * 16 + lg * 4 + r, col = v0 + j * 16 + ln;
                const float v = i < len && col < s.V ? load1<DT>(in.v.row(b, start + i, h), col) : 0.0f;
                y[r] = fmaf(-en[r], ks_[j][r], v);
            }
            store_planes(rt + (j * 16 + ln) * kTS + w * 16 + lg * 4, kTPlane, y);
        }
        __syncthreads();

        f32x4 x[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) x[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            if (ks == 0 || w >= 2) {
                const Frag<3> a = ti[ks].frag();
#pragma unroll
                for (int j = 0; j < CT; ++j) mma(x[j], a, row_frag<3>(rt, kTPlane, kTS, j * 16, ks * 32, lane));
            }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            uint16_t* o = ut + (j * 16 + ln) * kTS + w * 16 + lg * 4;
            f32x4 u, l;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                u[r] = be[r] * x[j][r];
                l[r] = le[r] * u[r];
            }
            if (!KEEP) store_planes(o, kTPlane, u);
            store_planes(o + 3 * kTPlane, kTPlane, l);
        }
        __syncthreads();

#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int col = v0 + j * 16 + ln;
            if (KEEP) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = w * 16 + lg * 4 + r;
                    if (i < len && col < s.V) keep.x[(bh * s.T + start + i) * s.V + col] = x[j][r];
                }
            } else {
                f32x4 o = {0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    if (ks == 0 || w >= 2)
                        mma(o, at[ks].frag(), row_frag<3>(ut, kTPlane, kTS, j * 16, ks * 32, lane));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = w * 16 + lg * 4 + r;
                    if (p.out && i < len && col < s.V)
                        put1<DT>(p.out, ((b * s.T + start + i) * s.H + h) * (int64_t)s.V + col,
                                         in.scale * fmaf(en[r], qs[j][r], o[r]));
                }
            }
        }
        const float end = enter[len - 1];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][j][r] *= end;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const Frag<NP> kf = col_frag<NP>(kt, kKPlane, KS, ks * 32, (w * RT + i) * 16, lane);
#pragma unroll
                for (int j = 0; j < CT; ++j) mma(S[i][j], kf, row_frag<3>(lt, kTPlane, kTS, j * 16, ks * 32, lane));
            }
        }
        __syncthreads();
    }
    if (!KEEP && p.last)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int d = (w * RT + i) * 16 + lg * 4 + r, col = v0 + j * 16 + ln;
                    if (d < s.K && col < s.V) p.last[(bh * s.K + d) * s.V + col] = S[i][j][r];
                }
}

// The walk back.  With P the outputs' weights, dS the gradient of the state
// that leaves a block and everything scaled as above,
//   dU = scale P^T dO + leave K dS,  R = (I + diag(beta) M)^-T dU  (the gradient
//   of beta (V - enter K S)),  dV = beta R,
//   dS' = end dS + Q^T (scale enter dO) - K^T (beta enter R).
template <int DT, int RT, int CT>
__global__ void __launch_bounds__(kThreads) delta_walk_back(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep,
                                                            DeltaBwd p, Kept keep, int groups, bool vec) {
    constexpr int NP = kPlanes<DT>;
    constexpr int KP = 64 * RT, KS = KP + 8;
    constexpr int W = CT * 16;
    constexpr int OS = W + 8;  // elements of an LDS row of dO
    constexpr int kKPlane = kC * KS, kSPlane = W * KS, kTPlane = W * kTS, kOPlane = kC * OS;
    constexpr int kWide = 3 * (kSPlane > 2 * kTPlane ? kSPlane : 2 * kTPlane);
    // fp32 tiles of K and Q together pass the LDS from 192 rows on: Q then takes K's place
    constexpr bool kShare = DT == DT_F32 && RT >= 2;
    __shared__ __attribute__((aligned(16))) uint16_t kt[NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t qt_[kShare ? 8 : NP * kKPlane];
    __shared__ __attribute__((aligned(16))) uint16_t wide[kWide];  // dS, then what goes into K^T and Q^T
    __shared__ __attribute__((aligned(16))) uint16_t rt[3 * kTPlane];
    __shared__ __attribute__((aligned(16))) uint16_t ot[NP * kOPlane];  // dO [token][column]
    __shared__ __attribute__((aligned(16))) float enter[kC], leave[kC], beta[kC];
    uint16_t *const lt = wide, *const et = wide + 3 * kTPlane;
    uint16_t* const qt = kShare ? kt : qt_;

    int64_t bh;
    int group;
    if (!my_head(s, groups, bh, group)) return;
    const int64_t b = bh / s.H;
    const int h = (int)(bh % s.H), hk = h / (s.H / s.HK);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, ln = lane & 15, lg = lane >> 4;
    const int v0 = group * W;
    const int64_t slots = state_slots(s.T);

    auto load_tile = [&](uint16_t* tile, const HeadRows& rows, int start, int len) {
        for (int i = threadIdx.x; i < kC * KP / 8; i += kThreads) {
            const int r = i / (KP / 8), q = i % (KP / 8) * 8;
            Raw8<DT> x;
            load8(x, rows.row(b, start + r, hk), r < len, q, s.K, vec);
            store_frag(tile + r * KS + q, kKPlane, x.frag());
        }
    };

    f32x4 S[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = (w * RT + i) * 16 + lg * 4 + r, col = v0 + j * 16 + ln;
                S[i][j][r] = p.grad_last && d < s.K && col < s.V ? p.grad_last[(bh * s.K + d) * s.V + col] : 0.0f;
            }
    const int n = blocks.count(b);
    for (int c = n - 1; c >= 0; --c) {
        int start, len;
        blocks.at(b, c, start, len);
        const int row = w * 16 + ln, next = start + len;
        // what leaves this block enters the next one, unless a segment starts there
        if (next < s.T && in.reset && in.reset[b * s.T + next]) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j) S[i][j] = f32x4{0, 0, 0, 0};
        } else {
            const int64_t slot = next < s.T ? next / kC : slots - 1;
            float* to = keep.ds + (bh * slots + slot) * s.K * s.V;
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int d = (w * RT + i) * 16 + lg * 4 + r, col = v0 + j * 16 + ln;
                        if (d < s.K && col < s.V) to[(int64_t)d * s.V + col] = S[i][j][r];
                    }
        }
        Raw8<DT_F32> ti[2], at[2];  // columns of the inverse and of the weights: tokens from this row's on
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int64_t o = (bh * s.T + start + row) * kC + ks * 32 + lg * 8;
            const bool ok = row < len && (ks == 1 || w < 2);
            load8(ti[ks], reinterpret_cast<const char*>(prep.inv_t + o), ok, 0, 8, true);
            load8(at[ks], reinterpret_cast<const char*>(prep.att_t + o), ok, 0, 8, true);
        }
        load_tile(kt, in.k, start, len);
        if (!kShare) load_tile(qt, in.q, start, len);
        for (int i = threadIdx.x; i < kC * W; i += kThreads) {
            const int r = i / W, q = i % W;
            float x = 0.0f;
            if (r < len && v0 + q < s.V)
                x = Elem<DT>::load1(p.grad_out, ((b * s.T + start + r) * s.H + h) * (int64_t)s.V + v0 + q);
            uint32_t hi, mid, lo;
            split2(x, 0.0f, hi, mid, lo);
            ot[r * OS + q] = (uint16_t)hi;
            if (NP == 3) ot[kOPlane + r * OS + q] = (uint16_t)mid, ot[2 * kOPlane + r * OS + q] = (uint16_t)lo;
        }
        if (threadIdx.x < kC) {
            const bool ok = threadIdx.x < len;
            const int64_t o = bh * s.T + start + threadIdx.x;
            enter[threadIdx.x] = ok ? prep.enter[o] : 0.0f;
            leave[threadIdx.x] = ok ? prep.leave[o] : 0.0f;
            beta[threadIdx.x] = ok ? *reinterpret_cast<const float*>(in.beta.row(b, start + threadIdx.x, h)) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j)
                store_planes(wide + (j * 16 + ln) * KS + (w * RT + i) * 16 + lg * 4, kSPlane, S[i][j]);
        __syncthreads();

        f32x4 kd[CT], po[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) kd[j] = po[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k0 = 0; k0 < KP; k0 += 32) {
            const Frag<NP> kf = row_frag<NP>(kt, kKPlane, KS, w * 16, k0, lane);
#pragma unroll
            for (int j = 0; j < CT; ++j) mma(kd[j], kf, row_frag<3>(wide, kSPlane, KS, j * 16, k0, lane));
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            if (ks == 1 || w < 2) {
                const Frag<3> a = at[ks].frag();
#pragma unroll
                for (int j = 0; j < CT; ++j) mma(po[j], a, col_frag<NP>(ot, kOPlane, OS, ks * 32, j * 16, lane));
            }
        const f32x4 en = *reinterpret_cast<const f32x4*>(enter + w * 16 + lg * 4);
        const f32x4 le = *reinterpret_cast<const f32x4*>(leave + w * 16 + lg * 4);
        const f32x4 be = *reinterpret_cast<const f32x4*>(beta + w * 16 + lg * 4);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = fmaf(le[r], kd[j][r], in.scale * po[j][r]);
            store_planes(rt + (j * 16 + ln) * kTS + w * 16 + lg * 4, kTPlane, y);
        }
        __syncthreads();

        f32x4 x[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) x[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            if (ks == 1 || w < 2) {
                const Frag<3> a = ti[ks].frag();
#pragma unroll
                for (int j = 0; j < CT; ++j) mma(x[j], a, row_frag<3>(rt, kTPlane, kTS, j * 16, ks * 32, lane));
            }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int col = v0 + j * 16 + ln;
            uint16_t* o = lt + (j * 16 + ln) * kTS + w * 16 + lg * 4;
            f32x4 l, e;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = w * 16 + lg * 4 + r;
                const float dv = be[r] * x[j][r];
                l[r] = -en[r] * dv;
                e[r] = in.scale * en[r] * element<NP>(ot + i * OS + j * 16 + ln, kOPlane);
                if (i < len && col < s.V) {
                    keep.r[(bh * s.T + start + i) * s.V + col] = x[j][r];
                    put1<DT>(p.grad_v, ((b * s.T + start + i) * s.H + h) * (int64_t)s.V + col, dv);
                }
            }
            store_planes(o, kTPlane, l);
            store_planes(o + 3 * kTPlane, kTPlane, e);
        }
        __syncthreads();

        const float end = enter[len - 1];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][j][r] *= end;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const Frag<NP> kf = col_frag<NP>(kt, kKPlane, KS, ks * 32, (w * RT + i) * 16, lane);
#pragma unroll
                for (int j = 0; j < CT; ++j) mma(S[i][j], kf, row_frag<3>(lt, kTPlane, kTS, j * 16, ks * 32, lane));
            }
        }
        if (kShare) {
            __syncthreads();
            load_tile(qt, in.q, start, len);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const Frag<NP> qf = col_frag<NP>(qt, kKPlane, KS, ks * 32, (w * RT + i) * 16, lane);
#pragma unroll
                for (int j = 0; j < CT; ++j) mma(S[i][j], qf, row_frag<3>(et, kTPlane, kTS, j * 16, ks * 32, lane));
            }
        __syncthreads();
    }
    if (p.grad_h0) {
        const bool cut = in.reset && in.reset[b * s.T];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int d = (w * RT + i) * 16 + lg * 4 + r, col = v0 + j * 16 + ln;
                    if (d < s.K && col < s.V) p.grad_h0[(bh * s.K + d) * s.V + col] = cut ? 0.0f : S[i][j][r];
                }
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

dim3 walk_grid(const DeltaShape& s, int groups) { return dim3((unsigned)((s.B * s.H + 7) / 8 * 8 * groups)); }

template <int DT, bool KEEP>
hipError_t walk(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaFwd& out,
                const Kept& keep, hipStream_t st) {
    const bool vec = rows_vec(s, in);
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, CT = kMaxCT<DT, RT>;
        const int groups = (s.V + CT * 16 - 1) / (CT * 16);
        delta_walk<DT, RT, CT, KEEP><<<walk_grid(s, groups), kThreads, 0, st>>>(s, in, blocks, prep, out, keep, groups, vec);
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
                     const Kept& keep, hipStream_t st) {
    const bool vec = rows_vec(s, in);
    return by_rows(s, [&](auto rt) {
        constexpr int RT = decltype(rt)::value, CT = kMaxCT<DT, RT>;
        const int groups = (s.V + CT * 16 - 1) / (CT * 16);
        delta_walk_back<DT, RT, CT><<<walk_grid(s, groups), kThreads, 0, st>>>(s, in, blocks, prep, p, keep, groups, vec);
        return hipGetLastError();
    });
}

hipError_t run_walk_back(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                         const DeltaBwd& p, const Kept& keep, hipStream_t st) {
    return s.dtype == DT_BF16 ? walk_back<DT_BF16>(s, in, blocks, prep, p, keep, st)
                              : walk_back<DT_F32>(s, in, blocks, prep, p, keep, st);
}

}  // namespace delta
}  // namespace lrscan
