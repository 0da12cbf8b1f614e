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
#include "delta_tile.hpp"
#include "delta_ws.hpp"

namespace lrscan {
namespace delta {

constexpr int kWide = 512;    // threads of a workgroup
constexpr int kVS = 32 + 8;   // elements of an LDS row of 32 columns
constexpr int kGS = kC + 8;   // of 64

// A wavefront has 16 of the block's tokens (wt) and half of the other side's tiles of 16 (wh).
template <int DT>
__global__ void __launch_bounds__(kWide) delta_grads(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaBwd p,
                                                     HeadRows go, Kept keep, int wk, int wv, int slots) {
    constexpr int NP = kPlanes<DT>;
    constexpr int kVPlane = kC * kVS, kTPlane = kC * kGS;
    // S (or X) and dS, 32 columns of 64 rows; in their place then 64 columns of K and Q
    constexpr int kOperands = 2 * (3 * kVPlane > NP * kTPlane ? 3 * kVPlane : NP * kTPlane);
    __shared__ __attribute__((aligned(16))) uint16_t ops[kOperands];
    __shared__ __attribute__((aligned(16))) uint16_t pt[3 * kTPlane], lt[3 * kTPlane];  // PD, LD [j][i]
    __shared__ __attribute__((aligned(16))) float enter[kC], leave[kC], beta[kC], gh[kC], gl[kC], dg[2 * kC];
    __shared__ float ends[kWide / 64];
    uint16_t *const st = ops, *const dt = ops + 3 * kVPlane, *const kb = ops, *const qb = ops + NP * kTPlane;
    const int lane = threadIdx.x & 63, w = wave_number(), ln = lane & 15, lg = lane >> 4;
    const int wt = w & 3, wh = w >> 2;
    const int64_t bk = blockIdx.x / slots, b = bk / s.HK;
    const int hk = (int)(bk % s.HK), share = s.H / s.HK;
    const int n = blocks.count(b);
    const int row = wt * 16 + ln;
    const int kw = kept_width(s.V);
    const int sr = threadIdx.x >> 3, sc = (threadIdx.x & 7) * 4;  // four columns of a staged row

    for (int c = blockIdx.x % slots; c < n; c += slots) {
        int start, len;
        bool first;
        blocks.at(b, c, start, len, first);
        const int next = start + len;
        const bool has_s = !first && (start > 0 || in.h0);
        bool cut = false;
        if (c + 1 < n) {
            int x, y;
            blocks.at(b, c + 1, x, y, cut);
        }
        const bool has_ds = next < s.T ? !cut : p.grad_last != nullptr;
        const int64_t nslots = state_slots(s.T);
        const Buffer krows = block_rows(in.k, b, hk, start, len), qrows = block_rows(in.q, b, hk, start, len);
        for (int hh = 0; hh < share; ++hh) {
            const int h = hk * share + hh;
            const int64_t bh = b * s.H + h, t0 = bh * s.T + start;
            const int64_t state = (int64_t)s.K * kw;
            const Buffer S = buffer(keep.s + (bh * nslots + start / kC) * state, has_s ? state * 4 : 0);
            const Buffer dS = buffer(keep.ds + (bh * nslots + (next < s.T ? next / kC : nslots - 1)) * state,
                                     has_ds ? state * 4 : 0);
            const Buffer orows = block_rows(go, b, h, start, len);
            const Buffer xrows = buffer(keep.x + t0 * kw, (int64_t)len * kw * 4);
            const Buffer rrows = buffer(keep.r + t0 * kw, (int64_t)len * kw * 4);

            // ---- products of tokens with tokens ----
            f32x4 dp[2], dl[2];  // tiles 2 i + wh of the other tokens
#pragma unroll
            for (int i = 0; i < 2; ++i) dp[i] = dl[i] = f32x4{0, 0, 0, 0};
            f32x4 xs = __builtin_bit_cast(f32x4, load16(xrows, sc < kw ? (sr * kw + sc) * 4 : kNowhere));
            Raw8<DT> o;
            Raw8<DT_F32> r;
            o.load(orows, row * (int)go.st, lg * 8, wv);
            r.load(rrows, row * kw * 4, lg * 8, kw);
            __syncthreads();
            if (threadIdx.x < kC) {
                const f32x4 g = __builtin_bit_cast(f32x4, load16(buffer(prep.gates + t0, len * 16), threadIdx.x * 16));
                enter[threadIdx.x] = g[0], leave[threadIdx.x] = g[1], beta[threadIdx.x] = g[2], gh[threadIdx.x] = g[3];
                gl[threadIdx.x] = load4(buffer(prep.gl + t0, len * 4), threadIdx.x * 4);
            }
            for (int v0 = 0; v0 < s.V; v0 += 32) {
                store_planes(st + sr * kVS + sc, kVPlane, xs);
                __syncthreads();
                const Frag<NP> of = o.frag();
                const Frag<3> rf = r.frag();
                const int v1 = v0 + 32;
                xs = __builtin_bit_cast(f32x4, load16(xrows, v1 + sc < kw ? (sr * kw + v1 + sc) * 4 : kNowhere));
                o.load(orows, row * (int)go.st, v1 + lg * 8, wv);
                r.load(rrows, row * kw * 4, v1 + lg * 8, kw);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (2 * i + wh <= wt) {
                        const Frag<3> xf = row_frag<3>(st, kVPlane, kVS, (2 * i + wh) * 16, 0, lane);
                        mma(dp[i], of, xf);
                        mma(dl[i], rf, xf);
                    }
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 2 * i + wh, col = j * 16 + ln;
                f32x4 pd = {0, 0, 0, 0}, ld = {0, 0, 0, 0};
                if (j <= wt) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = wt * 16 + lg * 4 + r;
                        if (col > t) continue;
                        const float d = beta[col] * expf((gh[t] - gh[col]) + (gl[t] - gl[col]));
                        pd[r] = in.scale * d * dp[i][r];
                        if (col < t)
                            ld[r] = -beta[t] * d * dl[i][r];
                        else if (t < len)
                            p.grad_beta[(b * s.T + start + t) * s.H + h] = dl[i][r];  // R_t . X_t
                    }
                }
                uint16_t* at = pt + col * kGS + wt * 16 + lg * 4;
                store_planes(at, kTPlane, pd);
                store_planes(lt + (at - pt), kTPlane, ld);
            }

            // ---- 64 columns of q and k at a time ----
            float dgi[4] = {0, 0, 0, 0}, end = 0.0f;
            for (int d0 = 0; d0 < s.K; d0 += 64) {
                Raw8<DT> kn, qn;
                {
                    const int r = threadIdx.x >> 3, q = d0 + (threadIdx.x & 7) * 8;
                    kn.load(krows, r * (int)in.k.st, q, wk);
                    qn.load(qrows, r * (int)in.q.st, q, wk);
                }
                f32x4 dq[2], kl[2], kr[2], kd[2];  // tiles 2 wh + j of the columns
#pragma unroll
                for (int j = 0; j < 2; ++j) dq[j] = kl[j] = kr[j] = kd[j] = f32x4{0, 0, 0, 0};
                f32x4 ss, ds;
                Raw8<DT_F32> x;
                auto load = [&](int v0) {
                    const uint32_t at = v0 + sc < kw ? ((d0 + sr) * kw + v0 + sc) * 4 : kNowhere;
                    ss = __builtin_bit_cast(f32x4, load16(S, at));
                    ds = __builtin_bit_cast(f32x4, load16(dS, at));
                    o.load(orows, row * (int)go.st, v0 + lg * 8, wv);
                    r.load(rrows, row * kw * 4, v0 + lg * 8, kw);
                    x.load(xrows, row * kw * 4, v0 + lg * 8, kw);
                };
                if (has_s || has_ds) {
                    load(0);
                    for (int v0 = 0; v0 < s.V; v0 += 32) {
                        __syncthreads();
                        float dot = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) dot = fmaf(ss[i], ds[i], dot);
                        end = fmaf(dot, enter[len - 1], end);
                        store_planes(st + sr * kVS + sc, kVPlane, ss);
                        store_planes(dt + sr * kVS + sc, kVPlane, ds);
                        __syncthreads();
                        const Frag<NP> of = o.frag();
                        const Frag<3> rf = r.frag(), xf = x.frag();
                        load(v0 + 32);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const Frag<3> sf = row_frag<3>(st, kVPlane, kVS, (2 * wh + j) * 16, 0, lane);
                            mma(dq[j], of, sf);
                            mma(kl[j], rf, sf);
                            mma(kd[j], xf, row_frag<3>(dt, kVPlane, kVS, (2 * wh + j) * 16, 0, lane));
                        }
                    }
                }
                __syncthreads();
                {
                    const int at = (threadIdx.x >> 3) * kGS + (threadIdx.x & 7) * 8;
                    store_frag(kb + at, kTPlane, kn.frag());
                    store_frag(qb + at, kTPlane, qn.frag());
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = wt * 16 + lg * 4 + r;
                        dq[j][r] *= in.scale * enter[t];
                        kl[j][r] *= -beta[t] * enter[t];
                        kd[j][r] *= leave[t] * beta[t];
                    }
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const bool low = ks == 0 || wt >= 2, high = ks == 1 || wt < 2;
                    Frag<NP> kf[2], qf[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        kf[j] = col_frag<NP>(kb, kTPlane, kGS, ks * 32, (2 * wh + j) * 16, lane);
                        qf[j] = col_frag<NP>(qb, kTPlane, kGS, ks * 32, (2 * wh + j) * 16, lane);
                    }
                    if (low) {
                        const Frag<3> a = col_frag<3>(pt, kTPlane, kGS, ks * 32, wt * 16, lane);
                        const Frag<3> l = col_frag<3>(lt, kTPlane, kGS, ks * 32, wt * 16, lane);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            mma(dq[j], a, kf[j]);
                            mma(kl[j], l, kf[j]);
                        }
                    }
                    if (high) {
                        const Frag<3> a = row_frag<3>(pt, kTPlane, kGS, wt * 16, ks * 32, lane);
                        const Frag<3> l = row_frag<3>(lt, kTPlane, kGS, wt * 16, ks * 32, lane);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            mma(kr[j], a, qf[j]);
                            mma(kr[j], l, kf[j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int lc = (2 * wh + j) * 16 + ln, col = d0 + lc;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = wt * 16 + lg * 4 + r;
                        const float k = element<NP>(kb + t * kGS + lc, kTPlane), q = element<NP>(qb + t * kGS + lc, kTPlane);
                        dgi[r] = fmaf(q, dq[j][r], dgi[r]);
                        dgi[r] = fmaf(k, kl[j][r] - (kr[j][r] + kd[j][r]), dgi[r]);
                        end = fmaf(k, kd[j][r], end);
                        if (t >= len || col >= s.K) continue;
                        const int64_t at = ((b * s.T + start + t) * s.HK + hk) * s.K + col;
                        float gq = dq[j][r], gk = kl[j][r] + (kr[j][r] + kd[j][r]);
                        if (hh) gq += keep.pq[at], gk += keep.pk[at];
                        if (hh + 1 < share) {
                            keep.pq[at] = gq, keep.pk[at] = gk;
                        } else {
                            put1<DT>(p.grad_q, at, gq);
                            put1<DT>(p.grad_k, at, gk);
                        }
                    }
                }
                __syncthreads();
            }
#pragma unroll
            for (int m = 1; m < 16; m *= 2)
#pragma unroll
                for (int r = 0; r < 4; ++r) dgi[r] += __shfl_xor(dgi[r], m);
#pragma unroll
            for (int m = 1; m < 64; m *= 2) end += __shfl_xor(end, m);
            if (ln == 0) *reinterpret_cast<f32x4*>(dg + wh * kC + wt * 16 + lg * 4) = f32x4{dgi[0], dgi[1], dgi[2], dgi[3]};
            if (lane == 0) ends[w] = end;
            __syncthreads();
            if (w == 0) {
                float x = lane < len ? dg[lane] + dg[kC + lane] : 0.0f;
                if (lane == len - 1)
                    x += ((ends[0] + ends[1]) + (ends[2] + ends[3])) + ((ends[4] + ends[5]) + (ends[6] + ends[7]));
#pragma unroll
                for (int m = 1; m < 64; m *= 2) {
                    const float y = __shfl_down(x, m);
                    if (lane + m < 64) x += y;
                }
                if (!has_s && lane == 0) x = 0.0f;  // nothing entered for it to decay
                if (lane < len) p.grad_g[(b * s.T + start + lane) * s.H + h] = x;
            }
        }
    }
}

template <int DT>
hipError_t grads(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep, const DeltaBwd& p,
                 const HeadRows& go, const Kept& keep, hipStream_t st) {
    const int slots = (int)((s.T + kC - 1) / kC);
    delta_grads<DT><<<dim3((unsigned)(s.B * s.HK * slots)), kWide, 0, st>>>(
        s, in, blocks, prep, p, go, keep, row_width(s.K, DT), row_width(s.V, DT), slots);
    return hipGetLastError();
}

hipError_t run_grads(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                     const DeltaBwd& p, const HeadRows& go, const Kept& keep, hipStream_t st) {
    return s.dtype == DT_BF16 ? grads<DT_BF16>(s, in, blocks, prep, p, go, keep, st)
                              : grads<DT_F32>(s, in, blocks, prep, p, go, keep, st);
}

}  // namespace delta
}  // namespace lrscan
