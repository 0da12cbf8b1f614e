// delta_grads.hip -- gated delta rule: the gradients of q, k, log_decay and
// beta, every block by itself once the walks have left the state S that enters
// it, the gradient dS of the one that leaves it, X and R (the gradient of
// beta (V - enter K S)).
//
// With U = beta X, D the decays between tokens, P = D o (Q K^T) and
//   PD = D o (scale dO U^T) (i >= j),  LD = -beta_i D o (R U^T) (i > j):
//   dQ  = scale enter dO S^T + PD K
//   dKl = -beta enter R S^T + LD K                    (k as the later token)
//   dKr = PD^T Q + LD^T K + leave U dS^T              (k as the earlier one)
//   dK  = dKl + dKr,  dbeta_i = R_i . X_i,
//   dG_i = q_i . dQ_i + k_i . (dKl_i - dKr_i), and at the block's last token
//   also <dS, S'>, S' the state that leaves; d log_decay_t = sum_{i >= t} dG_i.
// (q_i and the later k_i come with exp(G_i) everywhere, the earlier k with
// exp(-G_j), which gives dG from the three sums.)  A workgroup takes the heads
// that share its query/key head in turn, so their sums have a fixed order.
//
// A wavefront has 16 columns of q and k, and with them 16 rows of S and dS, which
// are operands as they lie in memory; what all of them need (dO, R and X, 64
// columns at a time, then PD, LD, K and Q) lies in LDS.  The products of tokens
// with tokens are spread over the wavefronts a tile of 16x16 at a time while the
// same columns are there.
//
// bf16 [8, 2048], 20 heads of 128 over 10 keys: 566 us, of which the matrix cores
// are busy for 103 (with both sums over heads in memory, 210 MB more to write and
// read, it takes 15 us more).  One workgroup a compute unit (LDS and registers allow
// no second one), whose two wavefronts a SIMD wait half of the time.  The next head's
// operands loaded ahead cost registers that spill (786 us), as K and Q kept in LDS for
// all heads (670).
#include "delta_tile.hpp"
#include "delta_ws.hpp"

namespace lrscan {
namespace delta {

constexpr int kGS = kC + 8;   // elements of an LDS row of 64
constexpr int kGPlane = kC * kGS;

template <int NA, int NB>
__device__ __forceinline__ void mma_pair(f32x4& c0, f32x4& c1, const Frag<NA> (&a)[2], const Frag<NB>& b) {
    f32x4 c[2] = {c0, c1};
    mma(c, a, b);
    c0 = c[0], c1 = c[1];
}

// TT: tiles of 16 tokens of a wavefront, 4, or 2 where K leaves half of the
// wavefronts without columns.
template <int DT, int TT>
__global__ void __launch_bounds__(kGradThreads, 2) delta_grads(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaBwd p,
                                                        HeadRows go, Kept keep, int wk, int wv, int slots) {
    constexpr int NP = kPlanes<DT>;
    constexpr int DN = 2 * TT;                       // tiles of columns of a workgroup
    constexpr int kKS = DN * 16 + 8, kKPlane = kC * kKS;
    constexpr int kRows = (6 + NP) * kGPlane;        // X, R, dO
    constexpr int kTiles = 2 * NP * kKPlane;         // then K and Q
    __shared__ __attribute__((aligned(16))) uint16_t ops[kRows > kTiles ? kRows : kTiles];
    __shared__ __attribute__((aligned(16))) uint16_t pt[3 * kGPlane], lt[3 * kGPlane];  // PD, LD [j][i]
    __shared__ __attribute__((aligned(16))) float gates[5 * kC];  // enter, leave, beta, G in two
    __shared__ __attribute__((aligned(16))) float dg[DN * kC];
    __shared__ float ends[kGradThreads / 64];
    // sums over the heads that share a q and k: as many of the two as there is room for here
    constexpr int kHeld = DT == DT_BF16 ? (TT == 2 ? 2 : 1) : TT == 2 ? 1 : 0;
    __shared__ f32x4 held[kHeld ? kHeld * TT * kGradThreads : 1];
    uint16_t *const xt = ops, *const rt = ops + 3 * kGPlane, *const ot = ops + 6 * kGPlane;
    uint16_t *const kb = ops, *const qb = ops + NP * kKPlane;
    const float *const enter = gates, *const leave = gates + kC, *const beta = gates + 2 * kC, *const gh = gates + 3 * kC,
                *const gl = gates + 4 * kC;
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int dt = w % DN, t0_ = w / DN * TT;  // the wavefront's tile of columns, and its first of tokens
    const int64_t bk = scalar((int)blockIdx.x / slots), b = scalar((int)bk / s.HK);
    const int hk = scalar((int)bk % s.HK), share = scalar(s.H / s.HK);
    const int n = blocks.count(b);
    const int kw = kept_width(s.V);
    const int sr = threadIdx.x >> 3, sc = (threadIdx.x & 7) * 8;  // eight columns of a staged row
    // tiles (i, j), j <= i, of the products of tokens with tokens: number w, and w + 8 of ten
    int ti[2], tj[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int x = w + 8 * q;
        ti[q] = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3;
        tj[q] = x - ti[q] * (ti[q] + 1) / 2;
    }

    // rows with more blocks than slots begin again at a slot of their own, so no XCD gets all of those
    for (int c = scalar((int)((blockIdx.x + bk) % slots)); c < n; c += slots) {
        int start, len;
        bool first;
        blocks.at(b, c, start, len, first);
        const int next = start + len;
        const bool has_s = !first && (start > 0 || in.h0);
        const bool cut = blocks.cut_behind(b, c, n);
        const bool has_ds = next < s.T ? !cut : p.grad_last != nullptr;
        const int64_t nslots = state_slots(s.T);
        const Buffer krows = block_rows(in.k, b, hk, start, len), qrows = block_rows(in.q, b, hk, start, len);
        for (int d0 = 0; d0 < s.K; d0 += 16 * DN) {
            const int col = d0 + dt * 16 + ln;
            const bool works = d0 + dt * 16 < s.K;
            // this thread's sums of q (n = 0) and k (1)
            auto sum = [&](int n, int i) -> f32x4& {
                return n < kHeld ? held[(n * TT + i) * kGradThreads + threadIdx.x]
                                 : keep.sums[((int64_t)blockIdx.x * 8 + n * TT + i) * kGradThreads + threadIdx.x];
            };
            for (int hh = 0; hh < share; ++hh) {
                const int h = hk * share + hh;
                const int64_t bh = b * s.H + h, t0 = bh * s.T + start;
                const int64_t state = (int64_t)s.K * kw;
                const Buffer S = buffer(keep.s + (bh * nslots + entering_slot(start)) * state, has_s ? state * 4 : 0);
                const Buffer dS = buffer(keep.ds + (bh * nslots + leaving_slot(s.T, next)) * state,
                                         has_ds ? state * 4 : 0);
                const Buffer orows = block_rows(go, b, h, start, len);
                const Buffer xrows = buffer(keep.x + t0 * kw, (int64_t)len * kw * 4);
                const Buffer rrows = buffer(keep.r + t0 * kw, (int64_t)len * kw * 4);
                Raw8<DT> o;
                Raw8<DT_F32> r, x;
                auto load = [&](int v0) {
                    o.load(orows, sr * (int)go.st, v0 + sc, wv);
                    r.load(rrows, sr * kw * 4, v0 + sc, kw);
                    x.load(xrows, sr * kw * 4, v0 + sc, kw);
                };
                const f32x4 g = __builtin_bit_cast(f32x4, load16(buffer(prep.gates + t0, len * 16),
                                                                 threadIdx.x < kC ? threadIdx.x * 16 : kNowhere));
                const float gll = load4(buffer(prep.gl + t0, len * 4), threadIdx.x < kC ? threadIdx.x * 4 : kNowhere);
                load(0);

                f32x4 dp[2], dl[2], dq[TT], kl[TT], kr[TT];
                float end = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) dp[i] = dl[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < TT; ++i) dq[i] = kl[i] = kr[i] = f32x4{0, 0, 0, 0};
                for (int v0 = 0; v0 < s.V; v0 += 64) {
                    Raw8<DT_F32> ss[2], es[2];  // this wavefront's rows of the states
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        ss[k].load(S, col * kw * 4, v0 + k * 32 + lg * 8, kw);
                        es[k].load(dS, col * kw * 4, v0 + k * 32 + lg * 8, kw);
                    }
                    __syncthreads();  // what stood there is read
                    if (v0 == 0 && threadIdx.x < kC) {
                        const int i = threadIdx.x;
                        gates[i] = g[0], gates[kC + i] = g[1], gates[2 * kC + i] = g[2], gates[3 * kC + i] = g[3];
                        gates[4 * kC + i] = gll;
                    }
                    store_frag(ot + sr * kGS + sc, kGPlane, o.frag());
                    store_frag(rt + sr * kGS + sc, kGPlane, r.frag());
                    store_frag(xt + sr * kGS + sc, kGPlane, x.frag());
                    __syncthreads();
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (q == 0 || w < 2) {
#pragma unroll
                            for (int k = 0; k < 64; k += 32) {
                                const Frag<3> f = row_frag<3>(xt, kGPlane, kGS, tj[q] * 16, k, lane);
                                mma(dp[q], row_frag<NP>(ot, kGPlane, kGS, ti[q] * 16, k, lane), f);
                                mma(dl[q], row_frag<3>(rt, kGPlane, kGS, ti[q] * 16, k, lane), f);
                            }
                        }
                    if (works && (has_s || has_ds)) {
                        const float whole = enter[len - 1];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float dot = 0.0f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) dot = fmaf(ss[k].a[i], es[k].a[i], fmaf(ss[k].b[i], es[k].b[i], dot));
                            // wavefronts that share columns count them once
                            if (t0_ == 0) end = fmaf(dot, whole, end);
                            const Frag<3> sf = ss[k].frag(), ef = es[k].frag();
#pragma unroll
                            for (int i = 0; i < TT; i += 2) {
                                Frag<3> a[2];
                                Frag<NP> e[2];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    a[j] = row_frag<3>(rt, kGPlane, kGS, (t0_ + i + j) * 16, k * 32, lane);
                                    e[j] = row_frag<NP>(ot, kGPlane, kGS, (t0_ + i + j) * 16, k * 32, lane);
                                }
                                mma_pair(kl[i], kl[i + 1], a, sf);
                                mma_pair(dq[i], dq[i + 1], e, sf);
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    a[j] = row_frag<3>(xt, kGPlane, kGS, (t0_ + i + j) * 16, k * 32, lane);
                                mma_pair(kr[i], kr[i + 1], a, ef);
                            }
                        }
                    }
                    load(v0 + 64);
                }
                Raw8<DT> kn[DN / 4], qn[DN / 4];
#pragma unroll
                for (int i = 0; i < DN / 4; ++i) {
                    const int at = i * kGradThreads + threadIdx.x, row = at / (DN * 2), q = at % (DN * 2) * 8;
                    kn[i].load(krows, row * (int)in.k.st, d0 + q, wk);
                    qn[i].load(qrows, row * (int)in.q.st, d0 + q, wk);
                }
                // PD and LD, columns of the earlier token; the tiles above the diagonal are not read
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (q == 0 || w < 2) {
                        const int j = tj[q] * 16 + ln;
                        f32x4 pd, ld;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = ti[q] * 16 + lg * 4 + e;
                            const float d = beta[j] * expf((gh[t] - gh[j]) + (gl[t] - gl[j]));
                            // a token past the block has no gates, so its d may be infinite
                            pd[e] = j <= t && t < len ? in.scale * d * dp[q][e] : 0.0f;
                            ld[e] = j < t && t < len ? -beta[t] * d * dl[q][e] : 0.0f;
                            if (j == t && t < len && d0 == 0) p.grad_beta[(b * s.T + start + t) * s.H + h] = dl[q][e];  // R_t . X_t
                        }
                        uint16_t* at = pt + j * kGS + ti[q] * 16 + lg * 4;
                        store_planes(at, kGPlane, pd);
                        store_planes(lt + (at - pt), kGPlane, ld);
                        // of the two tiles that an operand of 32 spans, the one above the diagonal
                        if (ti[q] == tj[q] && (ti[q] & 1)) {
                            at -= 16;
#pragma unroll
                            for (int e = 0; e < 3; ++e)
                                *reinterpret_cast<u32x2*>(at + e * kGPlane) = *reinterpret_cast<u32x2*>(lt + (at - pt) + e * kGPlane) =
                                    u32x2{0, 0};
                        }
                    }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < DN / 4; ++i) {
                    const int at = i * kGradThreads + threadIdx.x, row = at / (DN * 2), q = at % (DN * 2) * 8;
                    store_frag(kb + row * kKS + q, kKPlane, kn[i].frag());
                    store_frag(qb + row * kKS + q, kKPlane, qn[i].frag());
                }
                __syncthreads();
                f32x4 dgi[TT], tq[TT], tk[TT];
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    dgi[i] = tq[i] = tk[i] = f32x4{0, 0, 0, 0};
                    if (hh) tq[i] = sum(0, i), tk[i] = sum(1, i);
                }
                if (works) {
                    f32x4 kv[TT];
#pragma unroll
                    for (int i = 0; i < TT; ++i) {
                        const int t = (t0_ + i) * 16 + lg * 4;
                        const f32x4 en = *reinterpret_cast<const f32x4*>(enter + t), le = *reinterpret_cast<const f32x4*>(leave + t),
                                    be = *reinterpret_cast<const f32x4*>(beta + t);
                        kv[i] = read_values<NP>(kb, kKPlane, kKS, (t0_ + i) * 16, dt * 16, lane);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            dq[i][e] *= in.scale * en[e];
                            kl[i][e] *= -be[e] * en[e];
                            kr[i][e] *= le[e] * be[e];
                            end = fmaf(kv[i][e], kr[i][e], end);
                        }
                    }
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        const Frag<NP> kf = col_frag<NP>(kb, kKPlane, kKS, ks * 32, dt * 16, lane);
                        const Frag<NP> qf = col_frag<NP>(qb, kKPlane, kKS, ks * 32, dt * 16, lane);
#pragma unroll
                        for (int i = 0; i < TT; ++i) {
                            const int t = t0_ + i;
                            if (ks == 0 || t >= 2) {
                                mma(dq[i], col_frag<3>(pt, kGPlane, kGS, ks * 32, t * 16, lane), kf);
                                mma(kl[i], col_frag<3>(lt, kGPlane, kGS, ks * 32, t * 16, lane), kf);
                            }
                            if (ks == 1 || t < 2) {
                                mma(kr[i], row_frag<3>(pt, kGPlane, kGS, t * 16, ks * 32, lane), qf);
                                mma(kr[i], row_frag<3>(lt, kGPlane, kGS, t * 16, ks * 32, lane), kf);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < TT; ++i) {
                        const f32x4 qv = read_values<NP>(qb, kKPlane, kKS, (t0_ + i) * 16, dt * 16, lane);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            dgi[i][e] = sum16(fmaf(qv[e], dq[i][e], kv[i][e] * (kl[i][e] - kr[i][e])));
                            tq[i][e] += dq[i][e];
                            tk[i][e] += kl[i][e] + kr[i][e];
                        }
                    }
                    if (hh + 1 < share) {
#pragma unroll
                        for (int i = 0; i < TT; ++i) sum(0, i) = tq[i], sum(1, i) = tk[i];
                    } else {
                        store_tokens<DT, TT>(p.grad_q, b * s.T + start, len, s.HK, hk, s.K, t0_ * 16, col, lane, tq);
                        store_tokens<DT, TT>(p.grad_k, b * s.T + start, len, s.HK, hk, s.K, t0_ * 16, col, lane, tk);
                    }
                }
#pragma unroll
                for (int m = 1; m < 64; m *= 2) end += __shfl_xor(end, m);
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    if (ln == 0) *reinterpret_cast<f32x4*>(dg + dt * kC + (t0_ + i) * 16 + lg * 4) = dgi[i];
                if (lane == 0) ends[w] = end;
                __syncthreads();
                if (w == 0) {
                    float x = 0.0f;
#pragma unroll
                    for (int i = 0; i < DN; ++i) x += dg[i * kC + lane];
                    if (lane >= len) x = 0.0f;
                    if (lane == len - 1)
                        x += ((ends[0] + ends[1]) + (ends[2] + ends[3])) + ((ends[4] + ends[5]) + (ends[6] + ends[7]));
#pragma unroll
                    for (int m = 1; m < 64; m *= 2) {
                        const float y = __shfl_down(x, m);
                        if (lane + m < 64) x += y;
                    }
                    if (!has_s && lane == 0) x = 0.0f;  // nothing entered for it to decay
                    float* to = p.grad_g + (b * s.T + start + lane) * s.H + h;
                    if (lane < len) *to = d0 ? *to + x : x;  // of the columns before
                }
            }
        }
    }
}

template <int DT, int TT>
hipError_t grads(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaBwd& p,
                 const HeadRows& go, const Kept& keep, hipStream_t st) {
    const int slots = (int)((s.T + kC - 1) / kC);
    delta_grads<DT, TT><<<dim3((unsigned)(s.B * s.HK * slots)), kGradThreads, 0, st>>>(
        s, in, blocks, prep, p, go, keep, row_width(s.K, DT), row_width(s.V, DT), slots);
    return hipGetLastError();
}

hipError_t run_grads(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                     const DeltaBwd& p, const HeadRows& go, const Kept& keep, hipStream_t st) {
    if (s.K <= 64)
        return s.dtype == DT_BF16 ? grads<DT_BF16, 2>(s, in, blocks, prep, p, go, keep, st)
                                  : grads<DT_F32, 2>(s, in, blocks, prep, p, go, keep, st);
    return s.dtype == DT_BF16 ? grads<DT_BF16, 4>(s, in, blocks, prep, p, go, keep, st)
                              : grads<DT_F32, 4>(s, in, blocks, prep, p, go, keep, st);
}

}  // namespace delta
}  // namespace lrscan
