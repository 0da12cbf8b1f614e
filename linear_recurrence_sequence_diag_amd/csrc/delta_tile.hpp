// delta_tile.hpp -- device building blocks of the gated delta rule's blocks of
// tokens (gfx950).
//
// Products on the matrix cores.  A fp32 value is the sum of three bf16 values,
// each the rest of those before it, rounded (what is left is below 2^-26), so a
// product of two fp32 operands is six bf16 products of 16x16x32 with fp32 sums
// (those left out are below 2^-26 of it), and a product with a bf16 operand is
// three.  The fp32 matrix instruction has a sixteenth of the bf16 rate, so six
// are 2.7 times as fast, three 5.3 times.  An infinity or NaN gives NaN.
//
// Layouts of v_mfma_f32_16x16x32_bf16, lane l, ln = l & 15, lg = l >> 4:
//   A: row ln, k = 8 lg .. 8 lg + 7      B: column ln, the same k
//   C: column ln, rows 4 lg .. 4 lg + 3
// The order of k is free as long as A and B agree.  Where a lane's eight k are
// 4 lg .. 4 lg + 3 of one tile of 16 and the same of the next one, two tiles of C
// are, as they stand in their registers, a B operand with their rows as k: a
// chain of products needs no exchange between lanes.  place() is where an index
// stands in rows that hold their k in that order.
#pragma once

#include "device.hpp"
#include "delta.hpp"
#include "delta_blocks.hpp"

namespace lrscan {
namespace delta {

constexpr int kThreads = 256;       // of a workgroup of blocks' operands, and of the step
constexpr int kWalkThreads = 512;   // of the walks
constexpr int kGradThreads = 512;   // of the gradients
constexpr int kScanThreads = 1024;  // of the search for segment starts

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Where index i stands in rows of that order (groups of 32).
__host__ __device__ __forceinline__ constexpr int place(int i) {
    return (i & ~31) + (i >> 2 & 3) * 8 + (i >> 4 & 1) * 4 + (i & 3);
}

template <int NP>
struct Frag {
    u32x4 p[NP];
};

// bf16 planes that hold a stored element exactly
template <int DT>
constexpr int kPlanes = DT == DT_F32 ? 3 : 1;

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

// c += a b, the small parts first: the products of parts i and j with i + j <= 2
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& c, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < NA && s - i < NB) c = mfma(a.p[i], b.p[s - i], c);
}

// c[j] += a[j] b, the sums in turn: a product does not wait for the one before
template <int NA, int NB, int M>
__device__ __forceinline__ void mma(f32x4 (&c)[M], const Frag<NA> (&a)[M], const Frag<NB>& b) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < NA && s - i < NB)
#pragma unroll
                for (int j = 0; j < M; ++j) c[j] = mfma(a[j].p[i], b.p[s - i], c[j]);
}

// two floats as three pairs of bf16, each the rounded rest of those before it
__device__ __forceinline__ void split2(float x0, float x1, uint32_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = pack_bf16x2(x0, x1);
        if (i < 2) {
            x0 -= __uint_as_float(p[i] << 16);
            x1 -= __uint_as_float(p[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ Frag<3> split8(f32x4 a, f32x4 b) {
    Frag<3> f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t p[3], q[3];
        split2(a[2 * j], a[2 * j + 1], p);
        split2(b[2 * j], b[2 * j + 1], q);
#pragma unroll
        for (int i = 0; i < 3; ++i) f.p[i][j] = p[i], f.p[i][2 + j] = q[i];
    }
    return f;
}

// Four consecutive k of a column, into three planes `step` elements apart.
__device__ __forceinline__ void store_planes(uint16_t* at, int step, f32x4 v) {
    uint32_t p[3], q[3];
    split2(v[0], v[1], p);
    split2(v[2], v[3], q);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x2*>(at + i * step) = u32x2{p[i], q[i]};
}

// ---- rows in memory ----
// A buffer descriptor of `bytes` from p on (p and bytes uniform): loads past the
// end give zeros and stores past it do nothing, which is how a block's missing
// tokens, and columns past a row's end (offset kNowhere), are left out.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ Buffer buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
// The whole offset goes where the bounds check looks at it.
__device__ __forceinline__ u32x4 load16(Buffer r, uint32_t at) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
__device__ __forceinline__ float load4(Buffer r, uint32_t at) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
}
__device__ __forceinline__ void store4(Buffer r, uint32_t at, float x) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), r, at, 0, 0);
}

// A value that is the same in all lanes, as a scalar (a division leaves it in
// vector registers, and a buffer descriptor made from those takes a loop over the
// lanes for every access).
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
// The wavefront's number in its workgroup.
__device__ __forceinline__ int wave_number() { return scalar((int)(threadIdx.x >> 6)); }

// An offset formed anew for each block (`with`: something of the block's): sums of
// it would otherwise stay in registers through a walk's loop, 16 and more of them.
__device__ __forceinline__ uint32_t anew(uint32_t x, int64_t with) {
    asm("" : "+v"(x) : "s"((uint32_t)with));
    return x;
}

// The rows of one head of an operand that belong to a block.  Rows are whole
// aligned vectors of 16 bytes (others were copied into such).
__device__ __forceinline__ Buffer block_rows(const HeadRows& rows, int64_t b, int64_t head, int start, int len) {
    return buffer(rows.row(b, start, head), len * rows.st);
}

// ---- eight consecutive elements of a row ----
template <int DT>
struct Raw8;
template <>
struct Raw8<DT_BF16> {
    u32x4 w;
    __device__ __forceinline__ Frag<1> frag() const { return Frag<1>{{w}}; }
    // columns c .. c + 7 of a row of n at byte `row`
    __device__ __forceinline__ void load(Buffer r, uint32_t row, int c, int n) {
        w = load16(r, c < n ? row + 2 * c : kNowhere);
    }
};
template <>
struct Raw8<DT_F32> {
    f32x4 a, b;
    __device__ __forceinline__ Frag<3> frag() const { return split8(a, b); }
    __device__ __forceinline__ void load(Buffer r, uint32_t row, int c, int n) {
        a = __builtin_bit_cast(f32x4, load16(r, c < n ? row + 4 * c : kNowhere));
        b = __builtin_bit_cast(f32x4, load16(r, c + 4 < n ? row + 4 * c + 16 : kNowhere));
    }
};

template <int DT>
__device__ __forceinline__ float load1(const char* row, int c) {
    return Elem<DT>::load1(row, c);
}

// One element; neighbouring lanes' parts of a line meet in the L2.
template <int DT>
__device__ __forceinline__ void put1(void* base, int64_t i, float x) {
    if constexpr (DT == DT_F32)
        reinterpret_cast<float*>(base)[i] = x;
    else
        reinterpret_cast<uint16_t*>(base)[i] = f32_to_bf16_bits(x);
}

// ---- LDS tiles of bf16 planes [NP][rows][stride] ----
// An A (or B) operand whose row (column) and k run as the tile's rows and columns.
template <int NP>
__device__ __forceinline__ Frag<NP> row_frag(const uint16_t* tile, int plane, int stride, int row0, int k0, int lane) {
    Frag<NP> f;
    const uint16_t* at = tile + (row0 + (lane & 15)) * stride + k0 + (lane >> 4) * 8;
#pragma unroll
    for (int i = 0; i < NP; ++i) f.p[i] = *reinterpret_cast<const u32x4*>(at + i * plane);
    return f;
}

// One whose k run down the tile's rows: element [k][row] of the tile, read with
// the transposing LDS load, in which 16 lanes read four rows of 16 elements and
// get four rows of one column each.
template <int NP>
__device__ __forceinline__ Frag<NP> col_frag(const uint16_t* tile, int plane, int stride, int k0, int col0, int lane) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    Frag<NP> f;
    const uint16_t* at = tile + (k0 + (lane >> 4) * 8 + (lane >> 2 & 3)) * stride + col0 + (lane & 3) * 4;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + i * plane));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + i * plane + 4 * stride));
        const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
        f.p[i] = u32x4{x[0], x[1], y[0], y[1]};
    }
    return f;
}

// Four rows of a tile in a lane's column: rows row0 + 4 lg .. 4 lg + 3, columns
// col0 + (lane & 3) * step .. of four lanes each.
template <int NP>
__device__ __forceinline__ void read_rows(u32x2 (&x)[NP], const uint16_t* tile, int plane, int stride, int row0, int col0,
                                          int step, int lane) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const uint16_t* at = tile + (row0 + (lane >> 4) * 4 + (lane >> 2 & 3)) * stride + col0 + (lane & 3) * step;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        x[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + i * plane)));
}
// An operand with the tile's rows k0 .. k0 + 31 as k, and 16 of its columns.
template <int NP>
__device__ __forceinline__ Frag<NP> rows_frag(const uint16_t* tile, int plane, int stride, int k0, int col0, int step,
                                              int lane) {
    u32x2 x[NP], y[NP];
    read_rows<NP>(x, tile, plane, stride, k0, col0, step, lane);
    read_rows<NP>(y, tile, plane, stride, k0 + 16, col0, step, lane);
    Frag<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i) f.p[i] = u32x4{x[i][0], x[i][1], y[i][0], y[i][1]};
    return f;
}
// The same where the tile's columns stand in place().
template <int NP>
__device__ __forceinline__ Frag<NP> placed_rows_frag(const uint16_t* tile, int plane, int stride, int k0, int col_tile,
                                                     int lane) {
    return rows_frag<NP>(tile, plane, stride, k0, (col_tile >> 1) * 32 + (col_tile & 1) * 4, 8, lane);
}
// Four values of a column as floats.
template <int NP>
__device__ __forceinline__ f32x4 read_values(const uint16_t* tile, int plane, int stride, int row0, int col0, int lane) {
    u32x2 x[NP];
    read_rows<NP>(x, tile, plane, stride, row0, col0, 4, lane);
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = __uint_as_float(j & 1 ? x[0][j >> 1] & 0xffff0000u : x[0][j >> 1] << 16);
        if constexpr (NP == 3) {
            const float m = __uint_as_float(j & 1 ? x[1][j >> 1] & 0xffff0000u : x[1][j >> 1] << 16);
            const float l = __uint_as_float(j & 1 ? x[2][j >> 1] & 0xffff0000u : x[2][j >> 1] << 16);
            v[j] += m + l;
        }
    }
    return v;
}

template <int NP>
__device__ __forceinline__ void store_frag(uint16_t* at, int plane, const Frag<NP>& f) {
#pragma unroll
    for (int i = 0; i < NP; ++i) *reinterpret_cast<u32x4*>(at + i * plane) = f.p[i];
}

// A lane's column of N tiles of tokens, from the block's token row0 on, of a
// contiguous [tokens, heads, width] output; what lies past the block's len tokens
// or the row's columns is left out.
template <int DT, int N>
__device__ __forceinline__ void store_tokens(void* out, int64_t t0, int len, int heads, int h, int width, int row0, int col,
                                             int lane, const f32x4 (&x)[N]) {
    constexpr int E = Elem<DT>::bytes;
    const int64_t step = (int64_t)heads * width * E;
    const Buffer rows = buffer(static_cast<char*>(out) + t0 * step + (int64_t)h * width * E, len * step);
    const uint32_t at = anew(col < width ? (row0 + (lane >> 4) * 4) * (int)step + col * E : kNowhere, t0);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (DT == DT_F32)
                store4(rows, at + (i * 16 + r) * (int)step, x[i][r]);
            else
                __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_bits(x[i][r]), rows, at + (i * 16 + r) * (int)step, 0, 0);
        }
}

// The sum of a value over the 16 lanes of a column tile, in all of them.
__device__ __forceinline__ float sum16(float x) {
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, true));  // row_ror 8
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x124, 0xf, 0xf, true));
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x122, 0xf, 0xf, true));
    x += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x121, 0xf, 0xf, true));
    return x;
}

// What prepares the blocks for the walk over them, by token: [B, H, T] and rows of kC.
struct Prep {
    // of a token, with G the running sum of log_decay in the block: exp(G_i), exp(G_end - G_i), beta and
    // the upper float of G; the lower one (backward)
    f32x4* gates;
    float* gl;
    // rows of kC in three bf16 planes, [B, H, T][plane][kC], their columns in place():
    uint16_t *inv, *att;      // (I + N)^-1, N_ij = decay_ij k_i.k_j beta_j (i > j); decay_ij q_i.k_j
    uint16_t *att_t, *inv_t;  // backward: columns of decay_ij q_i.k_j, and of (I + diag(beta) M)^-1, M = N / beta_j
};

// the matrix-core product of two small fp32 LDS matrices: one 16x16 tile of A B, depth k
__device__ __forceinline__ f32x4 mm16(const float* A, int sa, const float* B, int sb, int k, int lane) {
    f32x4 c = {0, 0, 0, 0};
    const int ln = lane & 15, lg = lane >> 4;
    for (int i = 0; i < k; i += 4)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(A[ln * sa + i + lg], B[(i + lg) * sb + ln], c, 0, 0, 0);
    return c;
}

}  // namespace delta
}  // namespace lrscan
