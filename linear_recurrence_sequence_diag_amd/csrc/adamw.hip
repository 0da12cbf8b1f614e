// adamw.hip -- the AdamW update of many tensors in few launches.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,   g = grad_scale grad,
//   w <- w (1 - rate wd) - rate / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// A launch takes up to kTensors tensors, whose descriptors lie in the kernel's
// arguments (so a captured launch holds them); a workgroup finds its tensor by
// bisection over the tensors' first workgroups.  A wavefront takes groups of
// 256 elements, four neighbours a lane: an 8-bit group's scale is then one
// reduction over the wavefront.  Bytes bound it: 16 a weight of state in fp32,
// 4 in 8 bits, beside the weight's and the gradient's own.
//
// 8-bit states.  m is held as e4m3 times the group's largest magnitude / 448;
// of v the square root, whose range is half of v's in the exponent, the same
// way.  e4m3 rounds to 3 bits (half a step is 2^-4 of the value) down to 2^-9 of
// its scale; a root above zero is held as at least that smallest code, so a
// small v next to a large one never turns into a division by eps alone.  The
// weights are updated from the fp32 m and v of this step, before they are
// rounded.
#include "adamw.hpp"
#include "device.hpp"

#include <cmath>

namespace lrscan {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // groups of a wavefront, all loads issued first
constexpr int64_t kPerBlock = (int64_t)(kThreads / 64) * kUnroll * kAdamwGroup;
constexpr int kTensors = 56;
constexpr float kTop = 448.0f, kBottom = 0x1p-9f;  // of e4m3

struct List {
    lrscan_adamw_tensor t[kTensors];
    uint32_t first[kTensors + 1];  // workgroups before each tensor
    int n;
};

struct Factors {
    float b1, c1, b2, c2;   // c = 1 - b
    float keep, eps;        // 1 - rate wd
    float step1, root2;     // rate / (1 - b1^t), 1 / sqrt(1 - b2^t)
    double rate, beta1, beta2;
    const int64_t* step;    // device: step1 and root2 are formed from it
    const float* scale;
};

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ f4 load4(const void* p, int64_t i, int n, bool vec) {
    f4 x = {0, 0, 0, 0};
    if (vec && n == 4) {
        if constexpr (DT == DT_F32) {
            x = __builtin_nontemporal_load(reinterpret_cast<const f4*>(static_cast<const float*>(p) + i));
        } else {
            const u2 w = __builtin_nontemporal_load(reinterpret_cast<const u2*>(static_cast<const uint16_t*>(p) + i));
            x = f4{bf16_bits_to_f32(w[0] & 0xffff), bf16_bits_to_f32(w[0] >> 16), bf16_bits_to_f32(w[1] & 0xffff),
                   bf16_bits_to_f32(w[1] >> 16)};
        }
        return x;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) x[j] = Elem<DT>::load1(p, i + j);
    return x;
}

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, int n, bool vec, f4 x) {
    if (vec && n == 4) {
        if constexpr (DT == DT_F32) {
            __builtin_nontemporal_store(x, reinterpret_cast<f4*>(static_cast<float*>(p) + i));
        } else {
            const u2 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
            __builtin_nontemporal_store(w, reinterpret_cast<u2*>(static_cast<uint16_t*>(p) + i));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) Elem<DT>::store1(p, i + j, x[j]);
}

__device__ __forceinline__ uint32_t load_codes(const void* p, int64_t i, int n, bool vec) {
    const uint8_t* c = static_cast<const uint8_t*>(p) + i;
    if (vec && n == 4) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(c));
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) w |= (uint32_t)c[j] << (8 * j);
    return w;
}

__device__ __forceinline__ void store_codes(void* p, int64_t i, int n, bool vec, uint32_t w) {
    uint8_t* c = static_cast<uint8_t*>(p) + i;
    if (vec && n == 4) {
        __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(c));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) c[j] = (uint8_t)(w >> (8 * j));
}

__device__ __forceinline__ f4 decode(uint32_t w, float scale) {
    return f4{__builtin_amdgcn_cvt_f32_fp8(w, 0), __builtin_amdgcn_cvt_f32_fp8(w, 1),
              __builtin_amdgcn_cvt_f32_fp8(w, 2), __builtin_amdgcn_cvt_f32_fp8(w, 3)} * scale;
}

// A group's codes and, from lane 0, its scale.  Groups whose largest magnitude
// is below 2^-100 count as zero (its reciprocal would leave fp32).
template <bool ROOT>
__device__ __forceinline__ uint32_t encode(f4 x, float* scale) {
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int m = 1; m < 64; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
    const bool none = top < 0x1p-100f;
    const float by = none ? 0.0f : 1.0f / top * kTop;
    if ((threadIdx.x & 63) == 0) *scale = none ? 0.0f : top * (1.0f / kTop);
    x *= by;
    if (ROOT)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = x[j] > 0.0f && x[j] < kBottom ? kBottom : x[j];
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
}

template <int DT, bool SMALL, bool MASTER>
__global__ void __launch_bounds__(kThreads) adamw(List list, Factors f) {
    __shared__ float from_step[2];
    int at = 0;
    for (int hi = list.n; hi - at > 1;) {  // first[at] <= block < first[hi]
        const int mid = (at + hi) >> 1;
        if (blockIdx.x >= list.first[mid])
            at = mid;
        else
            hi = mid;
    }
    const lrscan_adamw_tensor t = list.t[at];
    if (f.step) {
        if (threadIdx.x == 0) {
            const double s = (double)*f.step;
            from_step[0] = (float)(f.rate / -expm1(s * log(f.beta1)));
            from_step[1] = (float)(1.0 / sqrt(-expm1(s * log(f.beta2))));
        }
        __syncthreads();
        f.step1 = from_step[0];
        f.root2 = from_step[1];
    }
    const float gs = f.scale ? *f.scale : 1.0f;
    const uintptr_t wide = DT == DT_F32 ? 15 : 7;
    bool vec = !((reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad)) & wide) &&
               !((reinterpret_cast<uintptr_t>(t.exp_avg) | reinterpret_cast<uintptr_t>(t.exp_avg_sq)) & (SMALL ? 3 : 15));
    if (MASTER) vec = vec && !(reinterpret_cast<uintptr_t>(t.master) & 15);

    const int lane = threadIdx.x & 63;
    const int64_t g0 = ((int64_t)(blockIdx.x - list.first[at]) * (kThreads / 64) + (threadIdx.x >> 6)) * kUnroll;
    f4 w[kUnroll], g[kUnroll], m[kUnroll], v[kUnroll];
    uint32_t mc[kUnroll], vc[kUnroll];
    float ms[kUnroll], vs[kUnroll];
    int n[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = (g0 + u) * kAdamwGroup + lane * 4;
        const int64_t left = t.n - i;
        n[u] = left >= 4 ? 4 : left > 0 ? (int)left : 0;
        if (MASTER)
            w[u] = load4<DT_F32>(t.master, i, n[u], vec);
        else
            w[u] = load4<DT>(t.param, i, n[u], vec);
        g[u] = load4<DT>(t.grad, i, n[u], vec);
        if (SMALL) {
            mc[u] = load_codes(t.exp_avg, i, n[u], vec);
            vc[u] = load_codes(t.exp_avg_sq, i, n[u], vec);
            const bool held = (g0 + u) * kAdamwGroup < t.n;
            ms[u] = held ? t.exp_avg_scale[g0 + u] : 0.0f;
            vs[u] = held ? t.exp_avg_sq_scale[g0 + u] : 0.0f;
        } else {
            m[u] = load4<DT_F32>(t.exp_avg, i, n[u], vec);
            v[u] = load4<DT_F32>(t.exp_avg_sq, i, n[u], vec);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if ((g0 + u) * kAdamwGroup >= t.n) break;  // the whole wavefront
        const int64_t i = (g0 + u) * kAdamwGroup + lane * 4;
        if (SMALL) {
            m[u] = decode(mc[u], ms[u]);
            const f4 r = decode(vc[u], vs[u]);
            v[u] = r * r;
        }
        const f4 x = g[u] * gs;
        m[u] = m[u] * f.b1 + x * f.c1;
        v[u] = v[u] * f.b2 + x * x * f.c2;
        f4 root;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            root[j] = sqrtf(v[u][j]);
            w[u][j] = w[u][j] * f.keep - f.step1 * m[u][j] / (root[j] * f.root2 + f.eps);
        }
        if (MASTER) store4<DT_F32>(t.master, i, n[u], vec, w[u]);
        store4<DT>(t.param, i, n[u], vec, w[u]);
        if (SMALL) {
            store_codes(t.exp_avg, i, n[u], vec, encode<false>(m[u], t.exp_avg_scale + g0 + u));
            store_codes(t.exp_avg_sq, i, n[u], vec, encode<true>(root, t.exp_avg_sq_scale + g0 + u));
        } else {
            store4<DT_F32>(t.exp_avg, i, n[u], vec, m[u]);
            store4<DT_F32>(t.exp_avg_sq, i, n[u], vec, v[u]);
        }
    }
}

template <int DT>
void enqueue(const List& list, const Factors& f, bool small, bool masters, hipStream_t st) {
    const dim3 grid(list.first[list.n]), block(kThreads);
    if (small)
        masters ? adamw<DT, true, true><<<grid, block, 0, st>>>(list, f)
                : adamw<DT, true, false><<<grid, block, 0, st>>>(list, f);
    else
        masters ? adamw<DT, false, true><<<grid, block, 0, st>>>(list, f)
                : adamw<DT, false, false><<<grid, block, 0, st>>>(list, f);
}

}  // namespace

hipError_t launch_adamw(const lrscan_adamw_tensor* tensors, int64_t count, int dtype, int state_bits, bool masters,
                        const AdamwArgs& a, hipStream_t st) {
    Factors f{};
    f.b1 = (float)a.beta1, f.c1 = (float)(1.0 - a.beta1);
    f.b2 = (float)a.beta2, f.c2 = (float)(1.0 - a.beta2);
    f.keep = (float)(1.0 - a.rate * a.weight_decay);
    f.eps = (float)a.eps;
    f.rate = a.rate, f.beta1 = a.beta1, f.beta2 = a.beta2;
    f.step = a.step_dev;
    f.scale = a.grad_scale;
    if (!a.step_dev) {
        f.step1 = (float)(a.rate / -std::expm1((double)a.step * std::log(a.beta1)));
        f.root2 = (float)(1.0 / std::sqrt(-std::expm1((double)a.step * std::log(a.beta2))));
    }
    for (int64_t from = 0; from < count;) {
        List list;
        list.n = 0;
        list.first[0] = 0;
        while (list.n < kTensors && from < count) {
            const lrscan_adamw_tensor& t = tensors[from];
            const int64_t blocks = (t.n + kPerBlock - 1) / kPerBlock;
            if (list.n && list.first[list.n] + blocks > ((int64_t)1 << 30)) break;
            list.t[list.n] = t;
            list.first[list.n + 1] = list.first[list.n] + (uint32_t)blocks;
            ++list.n;
            ++from;
        }
        if (dtype == DT_BF16)
            enqueue<DT_BF16>(list, f, state_bits == 8, masters, st);
        else
            enqueue<DT_F32>(list, f, state_bits == 8, masters, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lrscan
