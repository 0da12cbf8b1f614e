// logits.hip -- penalties of tokens seen, biases and a grammar's mask on logits.
//
// A workgroup takes a slice of one row's vocabulary.  It counts the row's
// history into LDS, one word an entry of the slice (the upper bit: seen in the
// prompt; the others: how often answered), so nothing is kept between calls and
// the counts do not depend on the order of the atomics; the history is short
// beside the logits and comes from the L2 for every slice but the first.  A
// biased entry's word holds the number of the first list entry that names it;
// that one alone adds, later entries of the same token behind it in their order.
// Then one pass over the slice.  Bytes of the logits bound large vocabularies,
// the walk along a long history small ones: bf16 [32, 262144] takes 16.2 us with all
// rules, 2048 tokens and 64 entries a row (8.8 with none, a copy 6.1), of which the
// tables' clearing and the history are what is more; fp32 [5, 4001] 6.4 us.
#include "device.hpp"
#include "logits.hpp"

namespace lrscan {
namespace {

constexpr int kThreads = 512;
constexpr int kSlice = 4096;
constexpr uint32_t kSeen = 0x80000000u, kNone = 0xffffffffu;

template <class I>
__device__ __forceinline__ int64_t clamped(const void* p, int64_t b, int64_t other, int64_t top) {
    const int64_t x = p ? (int64_t)static_cast<const I*>(p)[b] : other;
    return x < 0 ? 0 : x > top ? top : x;
}

// Four or eight elements at an address that is aligned to the element only.
template <int DT>
__device__ __forceinline__ RowVec<DT> load_vec(const char* p) {
    RowVec<DT> r;
    __builtin_memcpy(&r.w, p, 16);
    return r;
}

// A sum as it stands in `named`: never the word that means none.
__device__ __forceinline__ uint32_t bias_bits(float sum) {
    const uint32_t w = __float_as_uint(sum);
    return w == kNone ? 0x7fc00000u : w;
}

template <int DT, class I, bool COUNT, bool BIAS>
__global__ void __launch_bounds__(kThreads) logits(LogitsArgs a, int slices) {
    constexpr int N = Elem<DT>::V, PER = kSlice / N / kThreads;  // vectors of a thread
    __shared__ __attribute__((aligned(16))) uint32_t count[COUNT ? kSlice : 4];
    __shared__ __attribute__((aligned(16))) uint32_t named[BIAS ? kSlice : 4];
    __shared__ int listed[BIAS ? kThreads : 1];
    __shared__ float values[BIAS ? kThreads : 1];
    __shared__ int twice;
    const int64_t b = blockIdx.x / slices;
    const int64_t v0 = (int64_t)(blockIdx.x % slices) * kSlice;
    const int n = (int)(a.V - v0 < kSlice ? a.V - v0 : kSlice);
    const char* in = static_cast<const char*>(a.in) + (b * a.in_stride + v0) * Elem<DT>::bytes;
    char* out = static_cast<char*>(a.out) + (b * a.out_stride + v0) * Elem<DT>::bytes;
    const uint32_t* allowed = a.allowed ? a.allowed + b * ((a.V + 31) / 32) : nullptr;

    // the slice's logits and mask are on their way while the history is counted
    RowVec<DT> x[PER];
    uint32_t open[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = (k * kThreads + threadIdx.x) * N;
        if (i + N <= n) x[k] = load_vec<DT>(in + (int64_t)i * Elem<DT>::bytes);
        // N entries share a word of the mask: v0 and i are multiples of N
        open[k] = kNone;
        if (allowed && i < n) open[k] = allowed[(v0 + i) >> 5] >> ((v0 + i) & 31);
    }

    const float rep = COUNT && a.repetition ? a.repetition[b] : 1.0f;
    const float pres = COUNT && a.presence ? a.presence[b] : 0.0f;
    const float freq = COUNT && a.frequency ? a.frequency[b] : 0.0f;

    if (COUNT || BIAS) {
        // so are the first tokens of the history and the first entries of the list
        const I* ids = static_cast<const I*>(a.bias_ids) + b * a.K;
        const float* bias = a.bias + b * a.K;
        const int64_t length = COUNT ? clamped<I>(a.lengths, b, a.L, a.L) : 0;
        const int64_t prompt = COUNT ? clamped<I>(a.prompts, b, 0, a.L) : 0;
        const I* t = static_cast<const I*>(a.tokens) + b * a.token_stride;
        I id[4];
        auto tokens = [&](int64_t i0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) id[j] = i0 + j * kThreads < length ? t[i0 + j * kThreads] : I(-1);
        };
        tokens(threadIdx.x);
        I mine = -1;
        float value = 0.0f;
        if (BIAS && threadIdx.x < a.K) mine = ids[threadIdx.x], value = bias[threadIdx.x];
        for (int i = threadIdx.x * 4; i < kSlice; i += kThreads * 4) {
            if (COUNT) *reinterpret_cast<uint4*>(count + i) = make_uint4(0, 0, 0, 0);
            if (BIAS) *reinterpret_cast<uint4*>(named + i) = make_uint4(kNone, kNone, kNone, kNone);
        }
        if (threadIdx.x == 0) twice = 0;
        __syncthreads();
        if (COUNT)
            for (int64_t i0 = threadIdx.x; i0 < length; i0 += 4 * kThreads) {
                if (i0 >= kThreads) tokens(i0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t at = (int64_t)id[j] - v0;
                    if (id[j] < 0 || at < 0 || at >= n) continue;
                    if (i0 + j * kThreads < prompt)
                        atomicOr(&count[at], kSeen);
                    else
                        atomicAdd(&count[at], 1u);
                }
            }
        // an entry's list position stands at its token, the first one's where there are several
        if (BIAS)
            for (int64_t i = threadIdx.x; i < a.K; i += kThreads) {
                const int64_t at = (int64_t)(i < kThreads ? mine : ids[i]) - v0;
                if (at >= 0 && at < n && atomicMin(&named[at], (uint32_t)i) != kNone) twice = 1;
            }
        __syncthreads();
        if (BIAS) {
            if (twice && a.K <= kThreads) {
                // the first position's entry adds those behind it in order, from LDS
                const int64_t at = threadIdx.x < a.K ? (int64_t)mine - v0 : -1;
                const bool first = at >= 0 && at < n && named[at] == threadIdx.x;
                listed[threadIdx.x] = at >= 0 && at < n ? (int)at : -1;
                values[threadIdx.x] = value;
                __syncthreads();
                if (first) {
                    float sum = value;
#pragma unroll 4
                    for (int j = threadIdx.x + 1; j < (int)a.K; ++j) sum = listed[j] == (int)at ? sum + values[j] : sum;
                    named[at] = bias_bits(sum);
                }
            } else if (twice) {
                // a longer list in pieces, each token's sum so far standing in `named`
                for (int i = threadIdx.x; i < kSlice; i += kThreads) named[i] = kNone;
                for (int64_t i0 = 0; i0 < a.K; i0 += kThreads) {
                    const int64_t i = i0 + threadIdx.x, at = i < a.K ? (int64_t)ids[i] - v0 : -1;
                    const int here = at >= 0 && at < n ? (int)at : -1;
                    const float own = i < a.K ? bias[i] : 0.0f;
                    __syncthreads();  // the piece before is read
                    listed[threadIdx.x] = here;
                    values[threadIdx.x] = own;
                    __syncthreads();
                    bool first = here >= 0;
                    for (int j = 0; j < (int)threadIdx.x && first; ++j) first = listed[j] != here;
                    if (first) {
                        float sum = named[here] == kNone ? own : __uint_as_float(named[here]) + own;
                        for (int j = threadIdx.x + 1; j < kThreads; ++j) sum = listed[j] == here ? sum + values[j] : sum;
                        named[here] = bias_bits(sum);
                    }
                }
            } else {
                for (int64_t i = threadIdx.x; i < a.K; i += kThreads) {
                    const int64_t at = (int64_t)(i < kThreads ? mine : ids[i]) - v0;
                    if (at >= 0 && at < n) named[at] = bias_bits(i < kThreads ? value : bias[i]);
                }
            }
            __syncthreads();
        }
    }
    auto adjust = [&](float z, uint32_t c, uint32_t name) {
        if (c) {
            if (a.repetition) z = z > 0.0f ? z / rep : z * rep;
            const uint32_t times = c & ~kSeen;
            if (times) {
                z -= freq * (float)times;
                z -= pres;
            }
        }
        return name != kNone ? z + __uint_as_float(name) : z;
    };
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = (k * kThreads + threadIdx.x) * N;
        if (i + N <= n) {
            float y[N];
#pragma unroll
            for (int j = 0; j < N; ++j) y[j] = x[k].get(j);
            // whole words of the tables at a time; few entries stand in any of them
            uint32_t c[N], name[N], any = 0, least = kNone;
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                uint4 u = make_uint4(0, 0, 0, 0), v = make_uint4(kNone, kNone, kNone, kNone);
                if (COUNT) u = *reinterpret_cast<const uint4*>(count + i + j);
                if (BIAS) v = *reinterpret_cast<const uint4*>(named + i + j);
                c[j] = u.x, c[j + 1] = u.y, c[j + 2] = u.z, c[j + 3] = u.w;
                name[j] = v.x, name[j + 1] = v.y, name[j + 2] = v.z, name[j + 3] = v.w;
                any |= u.x | u.y | u.z | u.w;
                least &= v.x & v.y & v.z & v.w;
            }
            if (any != 0 || least != kNone)
#pragma unroll
                for (int j = 0; j < N; ++j) y[j] = adjust(y[j], c[j], name[j]);
#pragma unroll
            for (int j = 0; j < N; ++j) y[j] = open[k] >> j & 1 ? y[j] : -__builtin_inff();
            uint32_t w[4];
            if constexpr (DT == DT_F32) {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(y[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
            }
            __builtin_memcpy(out + (int64_t)i * Elem<DT>::bytes, w, 16);
        } else {
            for (int j = 0; i + j < n; ++j) {
                float y = Elem<DT>::load1(in, i + j);
                y = adjust(y, COUNT ? count[i + j] : 0, BIAS ? named[i + j] : kNone);
                y = open[k] >> j & 1 ? y : -__builtin_inff();
                if constexpr (DT == DT_F32)
                    reinterpret_cast<float*>(out)[i + j] = y;
                else
                    reinterpret_cast<uint16_t*>(out)[i + j] = f32_to_bf16_bits(y);
            }
        }
    }
}

template <int DT, class I>
void enqueue(const LogitsArgs& a, hipStream_t st) {
    const int slices = (int)((a.V + kSlice - 1) / kSlice);
    const dim3 grid((unsigned)(a.B * slices)), block(kThreads);
    const bool count = a.tokens && (a.repetition || a.presence || a.frequency), bias = a.bias_ids != nullptr;
    if (count)
        bias ? logits<DT, I, true, true><<<grid, block, 0, st>>>(a, slices)
             : logits<DT, I, true, false><<<grid, block, 0, st>>>(a, slices);
    else
        bias ? logits<DT, I, false, true><<<grid, block, 0, st>>>(a, slices)
             : logits<DT, I, false, false><<<grid, block, 0, st>>>(a, slices);
}

template <int DT>
void by_ids(const LogitsArgs& a, hipStream_t st) {
    if (a.id_bytes == 4)
        enqueue<DT, int32_t>(a, st);
    else
        enqueue<DT, int64_t>(a, st);
}

}  // namespace

bool logits_fits(const LogitsArgs& a) {
    return a.V <= ((int64_t)1 << 31) - 32 && a.L <= ((int64_t)1 << 31) - 1 && a.K <= ((int64_t)1 << 31) - 1 &&
           a.B <= (((int64_t)1 << 32) / kThreads - 1) / ((a.V + kSlice - 1) / kSlice);  // work-items of the grid in 32 bits
}

hipError_t launch_logits(const LogitsArgs& a, hipStream_t st) {
    if (a.dtype == DT_BF16)
        by_ids<DT_BF16>(a, st);
    else
        by_ids<DT_F32>(a, st);
    return hipGetLastError();
}

}  // namespace lrscan
