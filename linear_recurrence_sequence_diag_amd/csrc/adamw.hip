// adamw.hip -- the AdamW update of many tensors in few launches.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,   g = grad_scale grad,
//   w <- w (1 - rate wd) - rate / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// A launch takes up to kTensors tensors, whose descriptors lie in the kernel's
// arguments (so a captured launch holds them); a workgroup finds its tensor by
// bisection over the tensors' first workgroups.  A lane takes four neighbours at a
// time, of 8-bit states eight: a group's 256 elements are then 32 lanes', its scale
// one reduction over them.  Bytes bound it: 16 a weight of state in fp32,
// 4 in 8 bits, beside the weight's and the gradient's own.  A workgroup's 4096
// elements are all in flight before the first is used: bf16 weights with fp32
// masters and states, 110 million, 525 us (5.9 TB/s); bf16 with 8-bit states
// 197 us (5.6 TB/s; a call after another 227 us, 273 with four elements a lane,
// whose loads and stores of codes are half as wide).
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

constexpr int kThreads = kAdamwThreads, kPerBlock = kAdamwPerBlock;
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

// E consecutive elements (4 or 8) in fours, from i on, n of them there; vec: in
// whole vectors.
template <int DT, int E>
__device__ __forceinline__ void load(f4 (&x)[E / 4], const void* p, int64_t i, int n, bool vec) {
    if (vec && n == E) {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int k = 0; k < E / 4; ++k)
                x[k] = __builtin_nontemporal_load(reinterpret_cast<const f4*>(static_cast<const float*>(p) + i + 4 * k));
        } else {
            typedef uint32_t words __attribute__((ext_vector_type(E / 2)));
            const words w = __builtin_nontemporal_load(reinterpret_cast<const words*>(static_cast<const uint16_t*>(p) + i));
#pragma unroll
            for (int j = 0; j < E; ++j)
                x[j / 4][j % 4] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) x[j / 4][j % 4] = j < n ? Elem<DT>::load1(p, i + j) : 0.0f;
}

template <int DT, int E>
__device__ __forceinline__ void store(void* p, int64_t i, int n, bool vec, const f4 (&x)[E / 4]) {
    if (vec && n == E) {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int k = 0; k < E / 4; ++k)
                __builtin_nontemporal_store(x[k], reinterpret_cast<f4*>(static_cast<float*>(p) + i + 4 * k));
        } else {
            typedef uint32_t words __attribute__((ext_vector_type(E / 2)));
            words w;
#pragma unroll
            for (int j = 0; j < E / 2; ++j) w[j] = pack_bf16x2(x[j / 2][2 * (j & 1)], x[j / 2][2 * (j & 1) + 1]);
            __builtin_nontemporal_store(w, reinterpret_cast<words*>(static_cast<uint16_t*>(p) + i));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (j < n) Elem<DT>::store1(p, i + j, x[j / 4][j % 4]);
}

// Eight codes.
__device__ __forceinline__ u2 load_codes(const void* p, int64_t i, int n, bool vec) {
    const uint8_t* c = static_cast<const uint8_t*>(p) + i;
    if (vec && n == 8) return __builtin_nontemporal_load(reinterpret_cast<const u2*>(c));
    u2 w = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) w[j / 4] |= (uint32_t)c[j] << (8 * (j & 3));
    return w;
}

__device__ __forceinline__ void store_codes(void* p, int64_t i, int n, bool vec, u2 w) {
    uint8_t* c = static_cast<uint8_t*>(p) + i;
    if (vec && n == 8) {
        __builtin_nontemporal_store(w, reinterpret_cast<u2*>(c));
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) c[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
}

__device__ __forceinline__ f4 decode(uint32_t w, float scale) {
    return f4{__builtin_amdgcn_cvt_f32_fp8(w, 0), __builtin_amdgcn_cvt_f32_fp8(w, 1),
              __builtin_amdgcn_cvt_f32_fp8(w, 2), __builtin_amdgcn_cvt_f32_fp8(w, 3)} * scale;
}

// The codes of a group of 32 lanes and, from its first one, its scale.  Groups
// whose largest magnitude is below 2^-100 count as zero (its reciprocal would
// leave fp32).
template <bool ROOT>
__device__ __forceinline__ u2 encode(f4 (&x)[2], float* scale) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j / 4][j % 4]));
#pragma unroll
    for (int m = 1; m < 32; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
    const bool none = top < 0x1p-100f;
    const float by = none ? 0.0f : 1.0f / top * kTop;
    if (scale && (threadIdx.x & 31) == 0) *scale = none ? 0.0f : top * (1.0f / kTop);
    u2 w;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        x[k] *= by;
        if (ROOT)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[k][j] = x[k][j] > 0.0f && x[k][j] < kBottom ? kBottom : x[k][j];
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[k][0], x[k][1], 0, false);
        w[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[k][2], x[k][3], lo, true);
    }
    return w;
}

template <int DT, bool SMALL, bool MASTER>
__global__ void __launch_bounds__(kThreads) adamw(List list, Factors f) {
    constexpr int E = SMALL ? 8 : 4, U = kPerBlock / kThreads / E;  // elements of a lane at a time, and times
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
    const uintptr_t wide = DT == DT_F32 || SMALL ? 15 : 7;
    bool vec = !((reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad)) & wide) &&
               !((reinterpret_cast<uintptr_t>(t.exp_avg) | reinterpret_cast<uintptr_t>(t.exp_avg_sq)) & (SMALL ? 7 : 15));
    if (MASTER) vec = vec && !(reinterpret_cast<uintptr_t>(t.master) & 15);

    const int lane = threadIdx.x & 63;
    const int64_t i0 = (int64_t)(blockIdx.x - list.first[at]) * kPerBlock + (int64_t)(threadIdx.x >> 6) * 64 * E * U + lane * E;
    f4 w[U][E / 4], g[U][E / 4], m[U][E / 4], v[U][E / 4];
    u2 mc[U], vc[U];
    float ms[U], vs[U];
    int n[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * 64 * E, left = t.n - i;
        n[u] = left >= E ? E : left > 0 ? (int)left : 0;
        if (MASTER)
            load<DT_F32, E>(w[u], t.master, i, n[u], vec);
        else
            load<DT, E>(w[u], t.param, i, n[u], vec);
        load<DT, E>(g[u], t.grad, i, n[u], vec);
        if constexpr (SMALL) {
            mc[u] = load_codes(t.exp_avg, i, n[u], vec);
            vc[u] = load_codes(t.exp_avg_sq, i, n[u], vec);
            const int64_t group = i / kAdamwGroup;
            const bool held = group * kAdamwGroup < t.n;
            ms[u] = held ? t.exp_avg_scale[group] : 0.0f;
            vs[u] = held ? t.exp_avg_sq_scale[group] : 0.0f;
        } else {
            load<DT_F32, E>(m[u], t.exp_avg, i, n[u], vec);
            load<DT_F32, E>(v[u], t.exp_avg_sq, i, n[u], vec);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * 64 * E;
        if (i - lane * E >= t.n) break;  // the whole wavefront
        f4 root[E / 4];
#pragma unroll
        for (int k = 0; k < E / 4; ++k) {
            if constexpr (SMALL) {
                m[u][k] = decode(mc[u][k], ms[u]);
                const f4 r = decode(vc[u][k], vs[u]);
                v[u][k] = r * r;
            }
            const f4 x = g[u][k] * gs;
            m[u][k] = m[u][k] * f.b1 + x * f.c1;
            v[u][k] = v[u][k] * f.b2 + x * x * f.c2;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                root[k][j] = sqrtf(v[u][k][j]);
                w[u][k][j] = w[u][k][j] * f.keep - f.step1 * m[u][k][j] / (root[k][j] * f.root2 + f.eps);
            }
        }
        if (MASTER) store<DT_F32, E>(t.master, i, n[u], vec, w[u]);
        store<DT, E>(t.param, i, n[u], vec, w[u]);
        if constexpr (SMALL) {
            const int64_t group = i / kAdamwGroup;
            const bool held = group * kAdamwGroup < t.n;
            store_codes(t.exp_avg, i, n[u], vec, encode<false>(m[u], held ? t.exp_avg_scale + group : nullptr));
            store_codes(t.exp_avg_sq, i, n[u], vec, encode<true>(root, held ? t.exp_avg_sq_scale + group : nullptr));
        } else {
            store<DT_F32, E>(t.exp_avg, i, n[u], vec, m[u]);
            store<DT_F32, E>(t.exp_avg_sq, i, n[u], vec, v[u]);
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
            if (list.first[list.n] + blocks > kAdamwMaxBlocks) break;
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
