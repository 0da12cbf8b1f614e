// quad.hpp -- four adjacent channels of a row as they are stored (8 or 16
// bytes), for kernels that keep more state for a channel than leaves room for
// eight bf16 channels a thread, or that have few rows to spread over the GPU.
#pragma once

#include "device.hpp"

namespace lrscan {

constexpr int kQuad = 4;

// FULL: rows are whole quads; then a quad is one access, whatever its address
// is aligned to, else the last one of a row goes channel by channel.
template <int DT>
struct Quad {
    static constexpr int S = Elem<DT>::bytes;
    static constexpr int W = DT == DT_F32 ? 4 : 2;  // dwords
    typedef unsigned int Raw __attribute__((ext_vector_type(W), aligned(S)));
    Raw w;
    __device__ __forceinline__ static Quad zero() {
        Quad q;
#pragma unroll
        for (int i = 0; i < W; ++i) q.w[i] = 0u;
        return q;
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (DT == DT_F32) return __uint_as_float(w[j]);
        else return (j & 1) ? __uint_as_float(w[j >> 1] & 0xffff0000u) : __uint_as_float(w[j >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[kQuad]) {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int j = 0; j < kQuad; ++j) w[j] = __float_as_uint(v[j]);
        } else {
            w[0] = pack_bf16x2(v[0], v[1]);
            w[1] = pack_bf16x2(v[2], v[3]);
        }
    }
    template <bool FULL>
    __device__ __forceinline__ static Quad load(const char* p, int nvalid) {
        Quad q = zero();
        if (FULL || nvalid == kQuad) {
            q.w = __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p));
        } else {
            float v[kQuad];
#pragma unroll
            for (int j = 0; j < kQuad; ++j) v[j] = j < nvalid ? Elem<DT>::load1(p, j) : 0.0f;
            q.set(v);
        }
        return q;
    }
    template <bool FULL>
    __device__ __forceinline__ void store(char* p, int nvalid) const {
        if (FULL || nvalid == kQuad) {
            __builtin_nontemporal_store(w, reinterpret_cast<Raw*>(p));
        } else {
#pragma unroll
            for (int j = 0; j < kQuad; ++j)
                if (j < nvalid) Elem<DT>::store1(p, j, get(j));
        }
    }
};

}  // namespace lrscan
