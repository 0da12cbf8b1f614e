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
// the walk along a long history small ones.
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

template <int DT, class I, bool COUNT, bool BIAS>
__global__ void __launch_bounds__(kThreads) logits(LogitsArgs a, int slices) {
    constexpr int N = Elem<DT>::V;
    __shared__ uint32_t count[COUNT ? kSlice : 1];
    __shared__ uint32_t named[BIAS ? kSlice : 1];
    __shared__ int twice;
    const int64_t b = blockIdx.x / slices;
    const int64_t v0 = (int64_t)(blockIdx.x % slices) * kSlice;
    const int n = (int)(a.V - v0 < kSlice ? a.V - v0 : kSlice);

    if (COUNT || BIAS) {
        for (int i = threadIdx.x; i < kSlice; i += kThreads) {
            if (COUNT) count[i] = 0;
            if (BIAS) named[i] = kNone;
        }
        if (threadIdx.x == 0) twice = 0;
        __syncthreads();
        if (COUNT) {
            const int64_t length = clamped<I>(a.lengths, b, a.L, a.L), prompt = clamped<I>(a.prompts, b, 0, a.L);
            const I* t = static_cast<const I*>(a.tokens) + b * a.token_stride;
            for (int64_t i = threadIdx.x; i < length; i += kThreads) {
                const int64_t x = (int64_t)t[i] - v0;
                if (x < 0 || x >= n) continue;
                if (i < prompt)
                    atomicOr(&count[x], kSeen);
                else
                    atomicAdd(&count[x], 1u);
            }
        }
        const I* ids = static_cast<const I*>(a.bias_ids) + b * a.K;
        const float* bias = a.bias + b * a.K;
        if (BIAS)
            for (int64_t i = threadIdx.x; i < a.K; i += kThreads) {
                const int64_t x = (int64_t)ids[i] - v0;
                if (x >= 0 && x < n) atomicMin(&named[x], (uint32_t)i);
            }
        __syncthreads();
        if (BIAS) {
            for (int64_t i = threadIdx.x; i < a.K; i += kThreads) {
                const int64_t x = (int64_t)ids[i] - v0;
                if (x >= 0 && x < n && named[x] != (uint32_t)i) twice = 1;
            }
            __syncthreads();
            const bool again = twice != 0;
            // an owner replaces its number by the sum; the others' test against it is behind them
            for (int64_t i = threadIdx.x; i < a.K; i += kThreads) {
                const int64_t x = (int64_t)ids[i] - v0;
                if (x < 0 || x >= n) continue;
                bool first = true;
                if (again)
                    for (int64_t j = 0; j < i && first; ++j) first = ids[j] != ids[i];
                if (!first) continue;
                float sum = bias[i];
                if (again)
                    for (int64_t j = i + 1; j < a.K; ++j)
                        if (ids[j] == ids[i]) sum += bias[j];
                const uint32_t bits = __float_as_uint(sum);
                named[x] = bits == kNone ? 0x7fc00000u : bits;
            }
            __syncthreads();
        }
    }
    const float rep = COUNT && a.repetition ? a.repetition[b] : 1.0f;
    const float pres = COUNT && a.presence ? a.presence[b] : 0.0f;
    const float freq = COUNT && a.frequency ? a.frequency[b] : 0.0f;
    const uint32_t* allowed = a.allowed ? a.allowed + b * ((a.V + 31) / 32) : nullptr;
    auto adjust = [&](float z, int i, bool open) {
        if (COUNT) {
            const uint32_t c = count[i];
            if (c) {
                if (a.repetition) z = z > 0.0f ? z / rep : z * rep;
                const uint32_t times = c & ~kSeen;
                if (times) {
                    z -= freq * (float)times;
                    z -= pres;
                }
            }
        }
        if (BIAS && named[i] != kNone) z += __uint_as_float(named[i]);
        return open ? z : -__builtin_inff();
    };
    const char* in = static_cast<const char*>(a.in) + (b * a.in_stride + v0) * Elem<DT>::bytes;
    char* out = static_cast<char*>(a.out) + (b * a.out_stride + v0) * Elem<DT>::bytes;
    for (int i = threadIdx.x * N; i < n; i += kThreads * N) {
        // N entries share a word of the mask: v0 and i are multiples of N
        const uint32_t word = allowed ? allowed[(v0 + i) >> 5] >> ((v0 + i) & 31) : kNone;
        if (i + N <= n) {
            RowVec<DT> x = load_vec<DT>(in + (int64_t)i * Elem<DT>::bytes);
            float y[N];
#pragma unroll
            for (int j = 0; j < N; ++j) y[j] = adjust(x.get(j), i + j, word >> j & 1);
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
                const float y = adjust(Elem<DT>::load1(in, i + j), i + j, word >> j & 1);
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
           a.B <= ((int64_t)1 << 31) / ((a.V + kSlice - 1) / kSlice) - 1;
}

hipError_t launch_logits(const LogitsArgs& a, hipStream_t st) {
    if (a.dtype == DT_BF16)
        by_ids<DT_BF16>(a, st);
    else
        by_ids<DT_F32>(a, st);
    return hipGetLastError();
}

}  // namespace lrscan
