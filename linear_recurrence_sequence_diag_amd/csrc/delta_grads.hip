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

constexpr int kVS = 32 + 8;   // elements of an LDS row of 32 columns
constexpr int kTS2 = kC + 8;  // of 64

template <int DT>
__global__ void __launch_bounds__(kThreads) delta_grads(DeltaShape s, DeltaIn in, Blocks blocks, Prep prep, DeltaBwd p,
                                                        Kept keep, bool vec, bool vecv, int slots) {
    constexpr int NP = kPlanes<DT>;
    constexpr int kVPlane = kC * kVS, kTPlane = kC * kTS2;
    __shared__ __attribute__((aligned(16))) uint16_t st[3 * kVPlane], dt[3 * kVPlane];   // S (or X) and dS
    __shared__ __attribute__((aligned(16))) uint16_t pt[3 * kTPlane], lt[3 * kTPlane];   // PD, LD [j][i]
    __shared__ __attribute__((aligned(16))) uint16_t kb[NP * kTPlane], qb[NP * kTPlane]; // 64 columns of K, Q
    __shared__ __attribute__((aligned(16))) float enter[kC], leave[kC], beta[kC], gh[kC], gl[kC], dg[kC];
    __shared__ float ends[kThreads / 64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, ln = lane & 15, lg = lane >> 4;
    const int64_t bk = blockIdx.x / slots, b = bk / s.HK;
    const int hk = (int)(bk % s.HK), share = s.H / s.HK;
    const int n = blocks.count(b);
    const int row = w * 16 + ln;
    const bool vecx = s.V % 4 == 0;

    for (int c = blockIdx.x % slots; c < n; c += slots) {
        int start, len;
        blocks.at(b, c, start, len);
        const int next = start + len;
        const bool first = in.reset && in.reset[b * s.T + start];
        const bool has_s = !first && (start > 0 || in.h0);
        const bool has_ds = next < s.T ? !(in.reset && in.reset[b * s.T + next]) : p.grad_last != nullptr;
        const int64_t nslots = state_slots(s.T);
        for (int hh = 0; hh < share; ++hh) {
            const int h = hk * share + hh;
            const int64_t bh = b * s.H + h, t0 = bh * s.T + start;
            const float* S = keep.s + (bh * nslots + start / kC) * s.K * s.V;
            const float* dS = keep.ds + (bh * nslots + (next < s.T ? next / kC : nslots - 1)) * s.K * s.V;
            const char* go = static_cast<const char*>(p.grad_out) +
                             ((b * s.T + start + row) * s.H + h) * (int64_t)s.V * Elem<DT>::bytes;
            const char* rr = reinterpret_cast<const char*>(keep.r + (t0 + row) * s.V);
            const char* xr = reinterpret_cast<const char*>(keep.x + (t0 + row) * s.V);
            const bool ok = row < len;

            __syncthreads();
            if (threadIdx.x < kC) {
                const bool in_ = threadIdx.x < len;
                const int64_t o = t0 + threadIdx.x;
                enter[threadIdx.x] = in_ ? prep.enter[o] : 0.0f;
                leave[threadIdx.x] = in_ ? prep.leave[o] : 0.0f;
                gh[threadIdx.x] = in_ ? prep.gh[o] : 0.0f;
                gl[threadIdx.x] = in_ ? prep.gl[o] : 0.0f;
                beta[threadIdx.x] = in_ ? *reinterpret_cast<const float*>(in.beta.row(b, start + threadIdx.x, h)) : 0.0f;
            }

            // ---- products of tokens with tokens ----
            f32x4 dp[4], dl[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) dp[j] = dl[j] = f32x4{0, 0, 0, 0};
            float db = 0.0f;
            for (int v0 = 0; v0 < s.V; v0 += 32) {
                __syncthreads();
                {
                    const int r = threadIdx.x >> 2, q = (threadIdx.x & 3) * 8;
                    Raw8<DT_F32> x;
                    load8(x, reinterpret_cast<const char*>(keep.x + (t0 + r) * s.V), r < len, v0 + q, s.V, vecx);
                    store_frag(st + r * kVS + q, kVPlane, x.frag());
                }
                __syncthreads();
                Raw8<DT> o;
                Raw8<DT_F32> r, x;
                load8(o, go, ok, v0 + lg * 8, s.V, vecv);
                load8(r, rr, ok, v0 + lg * 8, s.V, vecx);
                load8(x, xr, ok, v0 + lg * 8, s.V, vecx);
#pragma unroll
                for (int e = 0; e < 8; ++e) db = fmaf(r.get(e), x.get(e), db);
                const Frag<NP> of = o.frag();
                const Frag<3> rf = r.frag();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j <= w) {
                        const Frag<3> xf = row_frag<3>(st, kVPlane, kVS, j * 16, 0, lane);
                        mma(dp[j], of, xf);
                        mma(dl[j], rf, xf);
                    }
            }
            db += __shfl_xor(db, 16);
            db += __shfl_xor(db, 32);
            if (lg == 0 && ok) p.grad_beta[(b * s.T + start + row) * s.H + h] = db;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = j * 16 + ln;
                f32x4 pd = {0, 0, 0, 0}, ld = {0, 0, 0, 0};
                if (j <= w) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = w * 16 + lg * 4 + r;
                        if (col > i) continue;
                        const float d = beta[col] * expf((gh[i] - gh[col]) + (gl[i] - gl[col]));
                        pd[r] = in.scale * d * dp[j][r];
                        if (col < i) ld[r] = -beta[i] * d * dl[j][r];
                    }
                }
                uint16_t* at = pt + col * kTS2 + w * 16 + lg * 4;
                store_planes(at, kTPlane, pd);
                store_planes(lt + (at - pt), kTPlane, ld);
            }

            // ---- 64 columns of q and k at a time ----
            float dgi[4] = {0, 0, 0, 0}, end = 0.0f;
            for (int d0 = 0; d0 < s.K; d0 += 64) {
                f32x4 dq[4], kl[4], kr[4], kd[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) dq[j] = kl[j] = kr[j] = kd[j] = f32x4{0, 0, 0, 0};
                __syncthreads();
                for (int i = threadIdx.x; i < kC * 8; i += kThreads) {
                    const int r = i >> 3, q = (i & 7) * 8;
                    Raw8<DT> x;
                    load8(x, in.k.row(b, start + r, hk), r < len, d0 + q, s.K, vec);
                    store_frag(kb + r * kTS2 + q, kTPlane, x.frag());
                    load8(x, in.q.row(b, start + r, hk), r < len, d0 + q, s.K, vec);
                    store_frag(qb + r * kTS2 + q, kTPlane, x.frag());
                }
                if (has_s || has_ds)
                    for (int v0 = 0; v0 < s.V; v0 += 32) {
                        __syncthreads();
                        {
                            const int r = threadIdx.x >> 2, q = (threadIdx.x & 3) * 8;
                            const bool in_ = d0 + r < s.K;
                            Raw8<DT_F32> a, e;
                            load8(a, reinterpret_cast<const char*>(S + (int64_t)(d0 + r) * s.V), in_ && has_s, v0 + q, s.V, vecx);
                            load8(e, reinterpret_cast<const char*>(dS + (int64_t)(d0 + r) * s.V), in_ && has_ds, v0 + q, s.V, vecx);
                            float dot = 0.0f;
#pragma unroll
                            for (int i = 0; i < 8; ++i) dot = fmaf(a.get(i), e.get(i), dot);
                            end = fmaf(dot, enter[len - 1], end);
                            store_frag(st + r * kVS + q, kVPlane, a.frag());
                            store_frag(dt + r * kVS + q, kVPlane, e.frag());
                        }
                        __syncthreads();
                        Raw8<DT> o;
                        Raw8<DT_F32> r, x;
                        load8(o, go, ok, v0 + lg * 8, s.V, vecv);
                        load8(r, rr, ok, v0 + lg * 8, s.V, vecx);
                        load8(x, xr, ok, v0 + lg * 8, s.V, vecx);
                        const Frag<NP> of = o.frag();
                        const Frag<3> rf = r.frag(), xf = x.frag();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const Frag<3> sf = row_frag<3>(st, kVPlane, kVS, j * 16, 0, lane);
                            mma(dq[j], of, sf);
                            mma(kl[j], rf, sf);
                            mma(kd[j], xf, row_frag<3>(dt, kVPlane, kVS, j * 16, 0, lane));
                        }
                    }
                else
                    __syncthreads();
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = w * 16 + lg * 4 + r;
                        dq[j][r] *= in.scale * enter[i];
                        kl[j][r] *= -beta[i] * enter[i];
                        kd[j][r] *= leave[i] * beta[i];
                    }
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const bool low = ks == 0 || w >= 2, high = ks == 1 || w < 2;
                    Frag<3> a, l, at, l2;
                    if (low) {
                        a = col_frag<3>(pt, kTPlane, kTS2, ks * 32, w * 16, lane);
                        l = col_frag<3>(lt, kTPlane, kTS2, ks * 32, w * 16, lane);
                    }
                    if (high) {
                        at = row_frag<3>(pt, kTPlane, kTS2, w * 16, ks * 32, lane);
                        l2 = row_frag<3>(lt, kTPlane, kTS2, w * 16, ks * 32, lane);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Frag<NP> kf = col_frag<NP>(kb, kTPlane, kTS2, ks * 32, j * 16, lane);
                        const Frag<NP> qf = col_frag<NP>(qb, kTPlane, kTS2, ks * 32, j * 16, lane);
                        if (low) {
                            mma(dq[j], a, kf);
                            mma(kl[j], l, kf);
                        }
                        if (high) {
                            mma(kr[j], at, qf);
                            mma(kr[j], l2, kf);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = d0 + j * 16 + ln;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = w * 16 + lg * 4 + r;
                        const float k = element<NP>(kb + i * kTS2 + j * 16 + ln, kTPlane);
                        const float q = element<NP>(qb + i * kTS2 + j * 16 + ln, kTPlane);
                        dgi[r] = fmaf(q, dq[j][r], dgi[r]);
                        dgi[r] = fmaf(k, kl[j][r] - (kr[j][r] + kd[j][r]), dgi[r]);
                        end = fmaf(k, kd[j][r], end);
                        if (i >= len || col >= s.K) continue;
                        const int64_t o = ((b * s.T + start + i) * s.HK + hk) * s.K + col;
                        float gq = dq[j][r], gk = kl[j][r] + (kr[j][r] + kd[j][r]);
                        if (hh) gq += keep.pq[o], gk += keep.pk[o];
                        if (hh + 1 < share) {
                            keep.pq[o] = gq, keep.pk[o] = gk;
                        } else {
                            put1<DT>(p.grad_q, o, gq);
                            put1<DT>(p.grad_k, o, gk);
                        }
                    }
                }
            }
#pragma unroll
            for (int m = 1; m < 16; m *= 2)
#pragma unroll
                for (int r = 0; r < 4; ++r) dgi[r] += __shfl_xor(dgi[r], m);
#pragma unroll
            for (int m = 1; m < 64; m *= 2) end += __shfl_xor(end, m);
            if (ln == 0) *reinterpret_cast<f32x4*>(dg + w * 16 + lg * 4) = f32x4{dgi[0], dgi[1], dgi[2], dgi[3]};
            if (lane == 0) ends[w] = end;
            __syncthreads();
            if (w == 0) {
                float x = lane < len ? dg[lane] : 0.0f;
                if (lane == len - 1) x += (ends[0] + ends[1]) + (ends[2] + ends[3]);
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
                 const Kept& keep, hipStream_t st) {
    const int slots = (int)((s.T + kC - 1) / kC);
    const bool vecv = (reinterpret_cast<uintptr_t>(p.grad_out) | (uintptr_t)(s.V * Elem<DT>::bytes)) % 16 == 0;
    delta_grads<DT><<<dim3((unsigned)(s.B * s.HK * slots)), kThreads, 0, st>>>(s, in, blocks, prep, p, keep,
                                                                             rows_vec(s, in), vecv, slots);
    return hipGetLastError();
}

hipError_t run_grads(const DeltaShape& s, const DeltaIn& in, const Blocks& blocks, const Prep& prep,
                     const DeltaBwd& p, const Kept& keep, hipStream_t st) {
    return s.dtype == DT_BF16 ? grads<DT_BF16>(s, in, blocks, prep, p, keep, st)
                              : grads<DT_F32>(s, in, blocks, prep, p, keep, st);
}

}  // namespace delta
}  // namespace lrscan
