// embed.hip -- the embedding lookup with scaling and its gradient by sorted
// tokens:
//
//   out[n] = scale W[ids[n]],     grad_W[v] = scale sum_{n: ids[n] = v} g[n]
//
// Ids outside [0, V) name no row: the lookup writes zeros for them and the
// gradient leaves them out.
//
// The gradient is a sum over tokens whose number for a row is anything from
// none to all of them, and its order has to be fixed for results to repeat.
//
//  * The tokens are sorted by id first, stably, with their positions: a radix
//    sort of digits of at most 10 bits, each pass one counting and one
//    scattering launch, or for up to 8192 tokens one launch in all.
//  * Most rows of a large table have no token, and writing their zeros is most
//    of the work.  It needs no sort, so the sort's launches do it: after the
//    few workgroups that sort come many that clear a share of the table, and
//    the sort's own time is hidden behind them.
//    (Up to 256 tokens are not sorted at all: each looks for its own row's
//    other tokens among them, and a row's first token adds them.)
//  * The sorted tokens are cut into chunks of equal length, whatever rows they
//    name.  A wavefront adds its chunk's tokens row by row in fp32 and writes
//    every row that lies inside the chunk.  A row that crosses a chunk's end
//    leaves partial sums, which one more launch adds in the chunks' order, a
//    fourth of them to a wavefront.  A token that the batch consists of to half
//    or wholly is a long such row: 16384 tokens into bf16 [262144, 2560], whose
//    most frequent holds 3% of them, 257 us, half of them one token 274, all of
//    them 289.
//
// Bound (MI355X, caches flushed): bytes.  Lookup, 16384 tokens of bf16 rows of
// 2560: 20 us, 84 MB written at 4.2 TB/s and a table's rows read as the caches
// hold them.  Gradient of as many tokens into bf16 [262144, 2560]: 254 us, of
// which some 203 are the four sort launches that write 1.34 GB of zeros on the
// side (6.6 TB/s; a fill reaches 6.9) and 51 the sums.  A small table's
// gradient is its launches: 6007 tokens into fp32 [4001, 1023] 14 us of sort,
// 10 of sums, 4 of crossing rows.
#include "embed.hpp"

#include <algorithm>

#include "device.hpp"
#include "launch.hpp"

namespace lrscan {

namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;
constexpr int kMaxDigitBits = 10;
constexpr int64_t kSortTile = 512;       // tokens a workgroup sorts, at least
constexpr int64_t kMaxSortBlocks = 256;  // then a workgroup takes more
constexpr int64_t kMaxChunks = 4096;     // chunks of sorted tokens (bounds the partial sums)
constexpr int kMinChunk = 16;

template <int IB>
__device__ __forceinline__ int64_t load_id(const void* ids, int64_t n) {
    if constexpr (IB == 8) return reinterpret_cast<const int64_t*>(ids)[n];
    else return reinterpret_cast<const int32_t*>(ids)[n];
}

// A thread's part of the rows: V columns from `at`.  The last vector of a row
// that is not whole vectors starts at D - V, so that it is whole too; the
// columns before `d0` are then also its neighbour's, who computes the same
// bits for them (lane by lane tests at every load made the f32 sums over rows
// of 1023 take 16.7 us against 9.7 for rows of 1024).  Rows shorter than a
// vector are read and written element by element.
template <int DT>
struct Columns {
    static constexpr int V = Elem<DT>::V;
    int64_t d0, at;  // first column that is the thread's own; first it computes
    bool some;       // it has any
    bool narrow;     // D < V
    bool blocks;     // rows written are whole 16-byte blocks: stored past the caches
    int n;           // columns of a narrow row
    __device__ __forceinline__ Columns(int64_t first, int64_t D, bool whole) {
        d0 = first;
        blocks = whole;
        some = d0 < D;
        narrow = D < V;
        n = narrow ? (int)D : V;
        at = narrow ? 0 : (d0 < D - V ? d0 : D - V);
    }
    __device__ __forceinline__ RowVec<DT> load(const void* base, size_t row, int64_t D) const {
        const size_t o = row * (size_t)D + (size_t)at;
        if (narrow) return load_row<DT, false>(base, o, n, 0.0f);
        RowVec<DT> r;
        r.w = load16_any(static_cast<const char*>(base) + o * Elem<DT>::bytes);
        return r;
    }
    __device__ __forceinline__ void store(void* base, size_t row, int64_t D, const RowOut<DT>& o, bool own) const {
        if (!some) return;
        char* q = static_cast<char*>(base) + (row * (size_t)D + (size_t)at) * Elem<DT>::bytes;
        if (blocks) {
            store16_nt(q, o.pack());
        } else if (!narrow && (!own || at == d0)) {
            store16_any(q, o.pack());
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n && at + j >= d0) Elem<DT>::store1(q, j, o.v[j]);
        }
    }
    __device__ __forceinline__ void load_floats(const float* row, float (&v)[V]) const {
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            if (narrow) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[q + j] = q + j < n ? row[q + j] : 0.0f;
            } else {
                const uint4 w = load16_any(row + at + q);
                v[q] = __uint_as_float(w.x);
                v[q + 1] = __uint_as_float(w.y);
                v[q + 2] = __uint_as_float(w.z);
                v[q + 3] = __uint_as_float(w.w);
            }
        }
    }
    __device__ __forceinline__ void store_floats(float* row, const float (&v)[V], bool own) const {
        if (!some) return;
        if (!narrow && (!own || at == d0)) {
#pragma unroll
            for (int q = 0; q < V; q += 4)
                store16_any(row + at + q, make_uint4(__float_as_uint(v[q]), __float_as_uint(v[q + 1]),
                                                     __float_as_uint(v[q + 2]), __float_as_uint(v[q + 3])));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n && at + j >= d0) row[at + j] = v[j];
        }
    }
};

// ---------------------------------------------------------------------------
// lookup: one thread to a 16-byte vector of an output row
// ---------------------------------------------------------------------------
template <int DT, int IB>
__global__ __launch_bounds__(kBlock) void embed_fwd_kernel(const void* __restrict__ ids,
                                                           const void* __restrict__ w, float scale,
                                                           void* __restrict__ out, int64_t N,
                                                           int64_t rows, int64_t D, bool blocks) {
    constexpr int V = Elem<DT>::V;
    // blockIdx.y counts groups of 64 vectors of a row, so a wavefront stays in one row
    const Columns<DT> col(((int64_t)blockIdx.y * kWave + threadIdx.x % kWave) * V, D, blocks);
    const int64_t n = (int64_t)blockIdx.x * kWaves + uniform((int)(threadIdx.x / kWave));
    if (n >= N || !col.some) return;
    const int64_t id = uniform64(load_id<IB>(ids, n));
    RowOut<DT> o;
    if (id >= 0 && id < rows) {
        const RowVec<DT> r = col.load(w, (size_t)id, D);
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = scale * r.get(j);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = 0.0f;
    }
    col.store(out, (size_t)n, D, o, false);
}

// ---------------------------------------------------------------------------
// stable radix sort of (id, position)
// ---------------------------------------------------------------------------
// The share of a table that one launch clears: 16-byte blocks [from, to) at
// `p`, and at the table's ends the bytes that are not whole blocks.
struct Clear {
    char* p;  // 16-byte aligned
    uint64_t from, to;
    char *head, *tail;
    uint32_t nhead, ntail;
};

// The workgroups of a launch past the first `first` clear, side by side, with
// their first kBlock threads each: half a workgroup's worth for every CU,
// writing one stretch of memory at a time.  Measured on MI355X, the gradient of
// 16384 tokens into bf16 [262144, 2560] with 16K, 32K, 48K, 64K and 128K threads:
// 255, 255, 267, 267 and 283 us; of 4000 into [262144, 1024]: 96, 94, 101, 97 and
// 109 (1.3 GB by 256K or 512K threads: 4.6 TB/s; non-temporal 6.3).
constexpr unsigned kClearThreads = 32768;
__device__ __forceinline__ void clear_share(const Clear& c, uint32_t first) {
    if (threadIdx.x >= kBlock) return;
    const uint64_t threads = (uint64_t)(gridDim.x - first) * kBlock;
    const uint64_t me = (uint64_t)(blockIdx.x - first) * kBlock + threadIdx.x;
    for (uint64_t i = c.from + me; i < c.to; i += threads)
        reinterpret_cast<uint4*>(c.p)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (me < c.nhead) c.head[me] = 0;
    if (me < c.ntail) c.tail[me] = 0;
}

struct SortPass {
    uint32_t N, tile, blocks;  // tokens; of one workgroup; workgroups that sort
    int shift, bits;
};

// Where a pass reads its keys: the ids themselves (an id that names no row is
// the key V, after every row), or what the pass before wrote.
template <int IB>
struct KeysFromIds {
    const void* ids;
    int64_t V;
    __device__ __forceinline__ uint32_t key(uint32_t n) const {
        const int64_t id = load_id<IB>(ids, n);
        return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
    }
    __device__ __forceinline__ uint32_t pos(uint32_t n) const { return n; }
};
struct KeysFromPass {
    const uint32_t *keys, *poss;
    __device__ __forceinline__ uint32_t key(uint32_t n) const { return keys[n]; }
    __device__ __forceinline__ uint32_t pos(uint32_t n) const { return poss[n]; }
};

// counts[block][digit]: tokens of the workgroup's tile with that digit.
template <class Src>
__global__ __launch_bounds__(kBlock) void sort_count_kernel(Src src, SortPass p, uint32_t* counts, Clear clear) {
    extern __shared__ uint32_t s_mem[];
    if (blockIdx.x >= p.blocks) {
        clear_share(clear, p.blocks);
        return;
    }
    const uint32_t digits = 1u << p.bits;
    for (uint32_t d = threadIdx.x; d < digits; d += kBlock) s_mem[d] = 0;
    __syncthreads();
    const uint64_t n0 = (uint64_t)blockIdx.x * p.tile;
    const uint64_t n1 = n0 + p.tile < p.N ? n0 + p.tile : p.N;
    for (uint64_t n = n0 + threadIdx.x; n < n1; n += kBlock)
        atomicAdd(&s_mem[(src.key((uint32_t)n) >> p.shift) & (digits - 1)], 1u);
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < digits; d += kBlock) counts[(size_t)blockIdx.x * digits + d] = s_mem[d];
}

// Every token of the tile to its place: the tokens of smaller digits, those of
// its digit in earlier workgroups, in earlier wavefronts of its own, and
// before it in its wavefront.  A wavefront owns consecutive tokens and ranks
// 64 at a time by the lanes that hold the same digit.
template <class Src>
__global__ __launch_bounds__(kBlock) void sort_scatter_kernel(Src src, SortPass p, const uint32_t* counts,
                                                              uint32_t* keys, uint32_t* poss, Clear clear) {
    extern __shared__ uint32_t s_mem[];  // next place of each digit, by wavefront
    __shared__ uint32_t s_wave[kWaves];
    if (blockIdx.x >= p.blocks) {
        clear_share(clear, p.blocks);
        return;
    }
    const uint32_t digits = 1u << p.bits;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const uint64_t n0 = (uint64_t)blockIdx.x * p.tile;
    const uint64_t n1 = n0 + p.tile < p.N ? n0 + p.tile : p.N;
    // this wavefront's tokens
    const uint64_t w0 = n0 + (uint64_t)wave * (p.tile / kWaves);
    const uint64_t w1 = w0 + p.tile / kWaves < n1 ? w0 + p.tile / kWaves : n1;
    uint32_t* mine = s_mem + (size_t)wave * digits;

    for (uint32_t d = tid; d < kWaves * digits; d += kBlock) s_mem[d] = 0;
    __syncthreads();
    for (uint64_t n = w0 + lane; n < w1; n += kWave)
        atomicAdd(&mine[(src.key((uint32_t)n) >> p.shift) & (digits - 1)], 1u);

    // places of the digits, four to a thread
    const uint32_t d = tid * 4;
    uint32_t total[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
    if (d < digits) {
        constexpr uint32_t U = 16;  // loads in flight (64 workgroups, 8-bit digits: 13 -> 11 us)
        for (uint32_t b0 = 0; b0 < p.blocks; b0 += U) {
            uint4 c[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                c[u] = *reinterpret_cast<const uint4*>(
                    counts + (size_t)(b0 + u < p.blocks ? b0 + u : p.blocks - 1) * digits + d);
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                const uint32_t cq[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t n = b0 + u < p.blocks ? cq[q] : 0u;
                    before[q] += b0 + u < blockIdx.x ? n : 0u;
                    total[q] += n;
                }
            }
        }
    }
    const uint32_t sum = total[0] + total[1] + total[2] + total[3];
    uint32_t upto = sum;  // inclusive over the wavefront, then over the workgroup
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t x = __shfl_up(upto, o, kWave);
        upto += lane >= (uint32_t)o ? x : 0u;
    }
    if (lane == kWave - 1) s_wave[wave] = upto;
    __syncthreads();  // (the counters above too)
    uint32_t base = upto - sum;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) base += w < wave ? s_wave[w] : 0u;
    if (d < digits) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t at = base + before[q];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = s_mem[(size_t)w * digits + d + q];
                s_mem[(size_t)w * digits + d + q] = at;
                at += c;
            }
            base += total[q];
        }
    }
    __syncthreads();
    // a wavefront's places are read and advanced by its own lanes only
    for (uint64_t m = w0; m < w1; m += kWave) {
        const uint64_t n = m + lane;
        const bool have = n < w1;
        const uint32_t key = have ? src.key((uint32_t)n) : 0;
        const uint32_t pos = have ? src.pos((uint32_t)n) : 0;
        const uint32_t digit = (key >> p.shift) & (digits - 1);
        unsigned long long same = __ballot(have);
        for (int b = 0; b < p.bits; ++b) {
            const unsigned long long one = __ballot((digit >> b) & 1u);
            same &= (digit >> b) & 1u ? one : ~one;
        }
        const unsigned long long below = same & ((1ull << lane) - 1);
        uint32_t at = 0;
        if (have) at = mine[digit] + (uint32_t)__popcll(below);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (have && below == 0) mine[digit] += (uint32_t)__popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (have) {
            keys[at] = key;
            poss[at] = pos;
        }
    }
}

// The whole sort in one workgroup, for up to kSmallTokens tokens whose key and
// position fit one word: the words stay in LDS and every pass moves them there
// (16 wavefronts of consecutive words, ranked as above).
constexpr int kSmallWaves = 16;
constexpr uint32_t kSmallTokens = 8192;
constexpr int kSmallBits = 8;
struct SmallSort {
    uint32_t N;
    int pos_bits, passes, bits;
};
template <class Src, int BITS>
__global__ __launch_bounds__(kSmallWaves* kWave) void sort_small_kernel(Src src, SmallSort p, uint32_t* keys,
                                                                        uint32_t* poss, Clear clear) {
    static_assert((1 << BITS) % kWave == 0, "the digits' places are whole wavefronts' work");
    constexpr int E = kSmallTokens / (kSmallWaves * kWave);
    __shared__ uint32_t s_word[kSmallTokens];
    __shared__ uint32_t s_at[kSmallWaves][1 << BITS];
    __shared__ uint32_t s_wave[4];
    if (blockIdx.x >= 1) {
        clear_share(clear, 1);
        return;
    }
    constexpr uint32_t digits = 1u << BITS;
    const uint32_t tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    // this thread's words: w0 + 64 e, e < rounds (whole rounds, shared evenly)
    const uint32_t rounds = (p.N + kSmallWaves * kWave - 1) / (kSmallWaves * kWave);
    const uint32_t w0 = wave * (rounds * kWave) + lane;
    uint32_t v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint32_t n = w0 + e * kWave;
        v[e] = (uint32_t)e < rounds && n < p.N ? (src.key(n) << p.pos_bits) | n : 0u;
    }
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = p.pos_bits + pass * BITS;
        for (uint32_t d = lane; d < digits; d += kWave) s_at[wave][d] = 0;
        // how many of the wavefront's words before this one have its digit
        uint32_t rank[E];
        unsigned long long same[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if ((uint32_t)e >= rounds) break;
            const uint32_t d = v[e] >> shift;
            same[e] = __ballot(w0 + e * kWave < p.N);
#pragma unroll
            for (int b = 0; b < BITS; ++b) {
                const unsigned long long one = __ballot((d >> b) & 1u);
                same[e] &= (d >> b) & 1u ? one : ~one;
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if ((uint32_t)e >= rounds) break;
            const uint32_t d = (v[e] >> shift) & (digits - 1);
            const unsigned long long below = same[e] & ((1ull << lane) - 1);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const uint32_t so_far = s_at[wave][d];
            rank[e] = so_far + (uint32_t)__popcll(below);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (w0 + e * kWave < p.N && below == 0) s_at[wave][d] = so_far + (uint32_t)__popcll(same[e]);
        }
        __syncthreads();
        // places of the digits, one to a thread
        uint32_t sum = 0, upto = 0;
        if (tid < digits) {
#pragma unroll
            for (int w = 0; w < kSmallWaves; ++w) sum += s_at[w][tid];
            upto = sum;
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) {
                const uint32_t x = __shfl_up(upto, o, kWave);
                upto += lane >= (uint32_t)o ? x : 0u;
            }
            if (lane == kWave - 1) s_wave[wave] = upto;
        }
        __syncthreads();
        if (tid < digits) {
            uint32_t at = upto - sum;
            for (uint32_t w = 0; w < wave; ++w) at += s_wave[w];
#pragma unroll
            for (int w = 0; w < kSmallWaves; ++w) {
                const uint32_t c = s_at[w][tid];
                s_at[w][tid] = at;
                at += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e)
            if ((uint32_t)e < rounds && w0 + e * kWave < p.N)
                s_word[s_at[wave][(v[e] >> shift) & (digits - 1)] + rank[e]] = v[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t n = w0 + e * kWave;
            v[e] = (uint32_t)e < rounds && n < p.N ? s_word[n] : 0u;
        }
        __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint32_t n = w0 + e * kWave;
        if ((uint32_t)e < rounds && n < p.N) {
            keys[n] = v[e] >> p.pos_bits;
            poss[n] = v[e] & ((1u << p.pos_bits) - 1);
        }
    }
}

// ---------------------------------------------------------------------------
// sums of the sorted tokens
// ---------------------------------------------------------------------------
struct Sorted {
    const uint32_t *keys, *poss;
    uint32_t N, V;       // a key of V names no row
    uint32_t chunk;      // tokens of a chunk (a power of two)
    float *head, *tail;  // [chunks, D] sums of rows that cross a chunk's start / end
    float scale;
    bool add;
    int64_t D;
    bool blocks;  // the table's rows are whole 16-byte blocks
};

// A finished row's vector: scaled, added to what is there if asked for, rounded.
template <int DT, int GDT>
__device__ __forceinline__ void put_row(const Sorted& s, void* grad, uint32_t row, const Columns<DT>& c,
                                        const float (&sum)[Elem<DT>::V]) {
    constexpr int V = Elem<DT>::V;
    if constexpr (GDT == DT) {
        RowOut<DT> o;
        if (s.add) {
            const RowVec<DT> old = c.load(grad, row, s.D);
#pragma unroll
            for (int j = 0; j < V; ++j) o.v[j] = fmaf(s.scale, sum[j], old.get(j));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) o.v[j] = s.scale * sum[j];
        }
        c.store(grad, row, s.D, o, s.add);
    } else {  // bf16 gradients into an fp32 table
        float* out = static_cast<float*>(grad) + (size_t)row * (size_t)s.D;
        float v[V];
        if (s.add) {
            c.load_floats(out, v);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = fmaf(s.scale, sum[j], v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = s.scale * sum[j];
        }
        c.store_floats(out, v, s.add);
    }
}

// One wavefront: one chunk, 64 vectors of the rows.
template <int DT, int GDT>
__global__ __launch_bounds__(kWave) void chunk_sum_kernel(Sorted s, const void* g, void* grad) {
    constexpr int V = Elem<DT>::V, U = 8;
    const uint32_t c = blockIdx.x, lane = threadIdx.x;
    const Columns<DT> col(((int64_t)blockIdx.y * kWave + lane) * V, s.D, s.blocks);
    const uint32_t p0 = c * s.chunk, p1 = s.N - p0 > s.chunk ? p0 + s.chunk : s.N;
    uint32_t cur = 0, after = s.V + 1;
    bool inside = false;  // the current row's first token lies in the chunk
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;

    // 32 tokens at a time: lane i holds the one at q0 - 1 + i, the token before
    // and the one after the batch too
    constexpr uint32_t kBatch = 32;
    for (uint32_t q0 = p0; q0 < p1; q0 += kBatch) {
        const uint32_t want = q0 + lane, n = p1 - q0 < kBatch ? p1 - q0 : kBatch;
        const uint32_t q = want == 0 ? 0 : (want - 1 < s.N ? want - 1 : s.N - 1);
        uint32_t key = 0, pos = 0;
        if (lane <= kBatch + 1) {
            key = s.keys[q];
            pos = s.poss[q];
        }
        const auto key_at = [&](uint32_t i) {  // of token q0 + i
            return (uint32_t)__builtin_amdgcn_readlane((int)key, (int)(i + 1));
        };
        if (q0 == p0) {
            cur = key_at(0);
            if (cur >= s.V) return;  // no row's tokens from here on
            inside = p0 == 0 || cur != (uint32_t)__builtin_amdgcn_readlane((int)key, 0);
        }
        if (p1 < s.N) after = key_at(n);
        for (uint32_t i0 = 0; i0 < n; i0 += U) {
            RowVec<DT> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {  // past the end: the last token again, not added
                const uint32_t at = i0 + u < n ? i0 + u : n - 1;
                const size_t row = (size_t)(uint32_t)__builtin_amdgcn_readlane((int)pos, (int)(at + 1));
                r[u] = col.load(g, row, s.D);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + u < n) {
                    const uint32_t k = key_at(i0 + u);
                    if (k != cur) {
                        if (inside) put_row<DT, GDT>(s, grad, cur, col, sum);
                        else col.store_floats(s.head + (size_t)c * s.D, sum, false);
                        if (k >= s.V) return;
                        cur = k;
                        inside = true;
#pragma unroll
                        for (int j = 0; j < V; ++j) sum[j] = 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] += r[u].get(j);
                }
            }
        }
    }
    if (!inside) col.store_floats(s.head + (size_t)c * s.D, sum, false);
    else if (after == cur) col.store_floats(s.tail + (size_t)c * s.D, sum, false);
    else put_row<DT, GDT>(s, grad, cur, col, sum);
}

// Up to kDirectTokens tokens, unsorted: one wavefront to a token and 64 vectors.
// The token's row is summed by its first token, in the order of positions.
constexpr uint32_t kDirectTokens = 256;
template <int DT, int GDT, class Src>
__global__ __launch_bounds__(kWave) void direct_sum_kernel(Sorted s, Src src, const void* g, void* grad) {
    constexpr int V = Elem<DT>::V, U = 8, Q = kDirectTokens / kWave;
    const uint32_t n = blockIdx.x, lane = threadIdx.x;
    uint32_t key[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const uint32_t t = q * kWave + lane;
        key[q] = t < s.N ? src.key(t) : s.V;
    }
    const uint32_t mine = uniform(src.key(n));
    if (mine >= s.V) return;
    unsigned long long same[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) same[q] = __ballot(key[q] == mine);
    uint32_t first = 0;
#pragma unroll
    for (int q = Q - 1; q >= 0; --q)
        if (same[q]) first = q * kWave + (uint32_t)__builtin_ctzll(same[q]);
    if (first != n) return;
    const Columns<DT> col(((int64_t)blockIdx.y * kWave + lane) * V, s.D, s.blocks);
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        while (same[q]) {  // eight rows at a time, the last one again in place of none
            RowVec<DT> r[U];
            uint32_t have = 0, at = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (same[q]) {
                    at = q * kWave + (uint32_t)__builtin_ctzll(same[q]);
                    same[q] &= same[q] - 1;
                    have = u + 1;
                }
                r[u] = col.load(g, at, s.D);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((uint32_t)u < have) {
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] += r[u].get(j);
                }
        }
    }
    put_row<DT, GDT>(s, grad, mine, col, sum);
}

__global__ __launch_bounds__(kBlock) void clear_kernel(Clear c) { clear_share(c, 0); }

// A row that starts in chunk c and goes on past it: the chunk's tail, then the
// heads of the chunks it runs through, a fourth of them to each wavefront.
template <int DT, int GDT>
__global__ __launch_bounds__(kBlock) void cross_sum_kernel(Sorted s, void* grad) {
    constexpr int V = Elem<DT>::V;
    __shared__ float s_sum[kWaves][kWave * V];
    const uint32_t c = blockIdx.x, lane = threadIdx.x % kWave;
    const uint32_t wave = uniform((int)(threadIdx.x / kWave));
    const uint32_t p0 = c * s.chunk, p1 = p0 + s.chunk;
    if (p1 >= s.N) return;
    const uint32_t start = p0 > 0 ? p0 - 1 : 0;
    const uint32_t k0 = uniform(s.keys[start]), k = uniform(s.keys[p1 - 1]), k1 = uniform(s.keys[p1]);
    if (k >= s.V || k1 != k) return;
    if (p0 > 0 && k0 == k) return;  // it started before
    // its last chunk: the first after c that ends with another key, looked for
    // 64 chunks at a time
    const uint32_t chunks = (s.N + s.chunk - 1) / s.chunk;
    uint32_t last = c + 1;
    for (;; last += kWave) {
        const uint32_t at = last + lane;
        bool ends = true;
        if (at + 1 < chunks) ends = s.keys[(at + 1) * s.chunk - 1] != k || s.keys[(at + 1) * s.chunk] != k;
        const unsigned long long found = __ballot(ends);
        if (found) {
            last += (uint32_t)__builtin_ctzll(found);
            break;
        }
    }
    const Columns<DT> col(((int64_t)blockIdx.y * kWave + lane) * V, s.D, s.blocks);
    const uint32_t per = (last - c + kWaves - 1) / kWaves;
    const uint32_t h0 = c + 1 + wave * per;
    const uint32_t h1 = h0 + per < last + 1 ? h0 + per : last + 1;
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    if (wave == 0) col.load_floats(s.tail + (size_t)c * s.D, sum);
    constexpr int U = 4;
    for (uint32_t h = h0; h < h1; h += U) {
        float v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) col.load_floats(s.head + (size_t)(h + u < h1 ? h + u : h1 - 1) * s.D, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += h + u < h1 ? v[u][j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s_sum[wave][lane * V + j] = sum[j];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += s_sum[w][lane * V + j];
    put_row<DT, GDT>(s, grad, k, col, sum);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool whole_blocks(const EmbedShape& s, const void* p) {
    const Shape c{s.N, 1, s.D, s.dtype};
    return rows_aligned(c, &p, 1);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct SortPlan {
    int passes, bits;
    uint32_t tile, blocks;
    uint32_t chunk, chunks;
    bool small;  // one launch sorts
    SmallSort one;
};

SortPlan sort_plan(const EmbedShape& s) {
    SortPlan p;
    int kb = 1;
    while (((int64_t)1 << kb) <= s.V) ++kb;  // keys 0 .. V
    p.passes = (kb + kMaxDigitBits - 1) / kMaxDigitBits;
    p.bits = std::max((kb + p.passes - 1) / p.passes, 2);  // a thread takes four digits at a time
    int pb = 1;
    while (((int64_t)1 << pb) < s.N) ++pb;
    p.small = s.N <= kSmallTokens && kb + pb <= 32;
    const int sp = (kb + kSmallBits - 1) / kSmallBits;
    p.one = SmallSort{(uint32_t)s.N, pb, sp, (kb + sp - 1) / sp};
    int64_t tile = (s.N + kMaxSortBlocks - 1) / kMaxSortBlocks;
    tile = (tile + kSortTile - 1) / kSortTile * kSortTile;
    p.tile = (uint32_t)tile;
    p.blocks = (uint32_t)((s.N + tile - 1) / tile);
    int64_t chunk = kMinChunk;
    while ((s.N + chunk - 1) / chunk > kMaxChunks) chunk *= 2;
    p.chunk = (uint32_t)chunk;
    p.chunks = (uint32_t)((s.N + chunk - 1) / chunk);
    return p;
}

struct EmbedWs {
    uint32_t *keys[2], *poss[2], *counts;
    float *head, *tail;
};

size_t ws_layout(const EmbedShape& s, void* base, EmbedWs* w) {
    const SortPlan p = sort_plan(s);
    char* c = static_cast<char*>(base);
    size_t at = 0;
    const auto take = [&](size_t words) {
        char* q = c + at;
        at += up256(words * 4);
        return q;
    };
    for (int i = 0; i < 2; ++i) {
        w->keys[i] = reinterpret_cast<uint32_t*>(take((size_t)s.N));
        w->poss[i] = reinterpret_cast<uint32_t*>(take((size_t)s.N));
    }
    w->counts = reinterpret_cast<uint32_t*>(take((size_t)p.blocks << p.bits));
    w->head = reinterpret_cast<float*>(take((size_t)p.chunks * s.D));
    w->tail = reinterpret_cast<float*>(take((size_t)p.chunks * s.D));
    return at;
}

// Shares of clearing a table of `bytes` bytes, one for each of `n` launches.
struct Clearing {
    char* table;
    uint64_t bytes;
    int n, done = 0;
    Clear next(unsigned* groups) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(table);
        const uint64_t nhead = std::min<uint64_t>((16 - at % 16) % 16, bytes);
        const uint64_t blocks = (bytes - nhead) / 16;
        Clear c;
        c.p = table + nhead;
        c.from = blocks / n * done;
        c.to = done + 1 == n ? blocks : blocks / n * (done + 1);
        c.head = table;
        c.nhead = done == 0 ? (uint32_t)nhead : 0u;
        c.tail = c.p + blocks * 16;
        c.ntail = done == 0 ? (uint32_t)(bytes - nhead - blocks * 16) : 0u;
        ++done;
        const uint64_t want = (c.to - c.from + kBlock - 1) / kBlock + (done == 1 ? 1 : 0);
        *groups = (unsigned)std::min<uint64_t>(want, kClearThreads / kBlock);
        if (bytes == 0) *groups = 0;
        return c;
    }
};

template <class Src>
hipError_t sort_pass(Src src, const SortPass& p, uint32_t* counts, uint32_t* keys, uint32_t* poss,
                     Clearing* clearing, hipStream_t st) {
    unsigned more = 0;
    Clear c = clearing->next(&more);
    hipLaunchKernelGGL((sort_count_kernel<Src>), dim3(p.blocks + more), dim3(kBlock), (size_t)4 << p.bits, st,
                       src, p, counts, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    c = clearing->next(&more);
    hipLaunchKernelGGL((sort_scatter_kernel<Src>), dim3(p.blocks + more), dim3(kBlock),
                       (size_t)(4 * kWaves) << p.bits, st, src, p, counts, keys, poss, c);
    return hipGetLastError();
}

template <class Src>
hipError_t sort_small(Src src, const SmallSort& p, uint32_t* keys, uint32_t* poss, Clearing* clearing,
                      hipStream_t st) {
    constexpr unsigned threads = kSmallWaves * kWave;
    unsigned more = 0;
    const Clear c = clearing->next(&more);
    if (p.bits <= 6)
        hipLaunchKernelGGL((sort_small_kernel<Src, 6>), dim3(1 + more), dim3(threads), 0, st, src, p, keys, poss, c);
    else
        hipLaunchKernelGGL((sort_small_kernel<Src, kSmallBits>), dim3(1 + more), dim3(threads), 0, st, src, p, keys,
                           poss, c);
    return hipGetLastError();
}

// The tokens sorted into keys[*at], poss[*at], and the table cleared.
template <class Src>
hipError_t sort_tokens(Src src, const SortPlan& plan, uint32_t N, const EmbedWs& w, char* table, uint64_t bytes,
                       int* at, hipStream_t st) {
    *at = 0;
    Clearing clearing{table, bytes, plan.small ? 1 : 2 * plan.passes};
    if (plan.small) return sort_small(src, plan.one, w.keys[0], w.poss[0], &clearing, st);
    SortPass p{N, plan.tile, plan.blocks, 0, plan.bits};
    hipError_t e = sort_pass(src, p, w.counts, w.keys[0], w.poss[0], &clearing, st);
    for (int i = 1; i < plan.passes && e == hipSuccess; ++i, *at ^= 1) {
        p.shift = i * plan.bits;
        e = sort_pass(KeysFromPass{w.keys[*at], w.poss[*at]}, p, w.counts, w.keys[*at ^ 1], w.poss[*at ^ 1],
                      &clearing, st);
    }
    return e;
}

template <int DT, int IB>
hipError_t embed_fwd_t(const EmbedShape& s, const void* ids, const void* w, float scale, void* out,
                       hipStream_t st) {
    const int64_t lanes = (int64_t)kWave * Elem<DT>::V;
    const dim3 grid((unsigned)((s.N + kWaves - 1) / kWaves), (unsigned)((s.D + lanes - 1) / lanes));
    hipLaunchKernelGGL((embed_fwd_kernel<DT, IB>), grid, dim3(kBlock), 0, st, ids, w, scale, out, s.N, s.V, s.D,
                       whole_blocks(s, out));
    return hipGetLastError();
}

template <int DT, int GDT>
hipError_t sums_t(const Sorted& x, uint32_t chunks, const void* g, void* grad, hipStream_t st) {
    const int64_t lanes = (int64_t)kWave * Elem<DT>::V;
    const uint32_t ncb = (uint32_t)((x.D + lanes - 1) / lanes);
    hipLaunchKernelGGL((chunk_sum_kernel<DT, GDT>), dim3(chunks, ncb), dim3(kWave), 0, st, x, g, grad);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || chunks == 1) return e;
    hipLaunchKernelGGL((cross_sum_kernel<DT, GDT>), dim3(chunks - 1, ncb), dim3(kBlock), 0, st, x, grad);
    return hipGetLastError();
}

// Without a sort: the table cleared, then the rows summed.
template <int DT, int GDT, class Src>
hipError_t direct_t(const Sorted& x, Src src, const void* g, void* grad, uint64_t bytes, hipStream_t st) {
    Clearing clearing{static_cast<char*>(grad), bytes, 1};
    unsigned groups = 0;
    const Clear c = clearing.next(&groups);
    if (groups > 0) {
        hipLaunchKernelGGL(clear_kernel, dim3(groups), dim3(kBlock), 0, st, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t lanes = (int64_t)kWave * Elem<DT>::V;
    hipLaunchKernelGGL((direct_sum_kernel<DT, GDT, Src>), dim3(x.N, (uint32_t)((x.D + lanes - 1) / lanes)),
                       dim3(kWave), 0, st, x, src, g, grad);
    return hipGetLastError();
}

template <class Src>
hipError_t direct(const EmbedShape& s, const Sorted& x, Src src, const void* g, void* grad, int grad_dtype,
                  uint64_t bytes, hipStream_t st) {
    if (s.dtype == DT_F32) return direct_t<DT_F32, DT_F32>(x, src, g, grad, bytes, st);
    if (grad_dtype == DT_F32) return direct_t<DT_BF16, DT_F32>(x, src, g, grad, bytes, st);
    return direct_t<DT_BF16, DT_BF16>(x, src, g, grad, bytes, st);
}

}  // namespace

bool embed_fits(const EmbedShape& s) {
    // 32-bit positions, keys and grid sizes (N below 2^26); a row's vectors, 64 at a time, along
    // the grid's second dimension (at most 65535)
    return s.N < ((int64_t)1 << 31) && s.V < ((int64_t)1 << 31) - 2 && s.D <= ((int64_t)1 << 23) &&
           (s.N + kWaves) / kWaves < ((int64_t)1 << 32) / kBlock;
}

hipError_t launch_embed_fwd(const EmbedShape& s, const void* ids, const void* w, float scale, void* out,
                            hipStream_t st) {
    if (s.dtype == DT_F32)
        return s.id_bytes == 8 ? embed_fwd_t<DT_F32, 8>(s, ids, w, scale, out, st)
                               : embed_fwd_t<DT_F32, 4>(s, ids, w, scale, out, st);
    return s.id_bytes == 8 ? embed_fwd_t<DT_BF16, 8>(s, ids, w, scale, out, st)
                           : embed_fwd_t<DT_BF16, 4>(s, ids, w, scale, out, st);
}

bool embed_sorts(const EmbedShape& s) { return s.N > kDirectTokens; }

size_t embed_ws_bytes(const EmbedShape& s) {
    EmbedWs w;
    return ws_layout(s, nullptr, &w);
}

hipError_t launch_embed_bwd(const EmbedShape& s, const void* ids, const void* g, float scale, void* grad,
                            int grad_dtype, bool add, void* ws, hipStream_t st) {
    const uint64_t row = (uint64_t)s.D * (grad_dtype == DT_F32 ? 4 : 2);
    const uint64_t bytes = add ? 0 : (uint64_t)s.V * row;
    char* table = static_cast<char*>(grad);
    if (!embed_sorts(s)) {
        const Sorted x{nullptr, nullptr, (uint32_t)s.N, (uint32_t)s.V, 0, nullptr, nullptr, scale, add, s.D,
                       whole_blocks(s, grad)};
        return s.id_bytes == 8 ? direct(s, x, KeysFromIds<8>{ids, s.V}, g, grad, grad_dtype, bytes, st)
                               : direct(s, x, KeysFromIds<4>{ids, s.V}, g, grad, grad_dtype, bytes, st);
    }
    EmbedWs w;
    ws_layout(s, ws, &w);
    const SortPlan plan = sort_plan(s);
    int at = 0;
    const hipError_t e =
        s.id_bytes == 8
            ? sort_tokens(KeysFromIds<8>{ids, s.V}, plan, (uint32_t)s.N, w, table, bytes, &at, st)
            : sort_tokens(KeysFromIds<4>{ids, s.V}, plan, (uint32_t)s.N, w, table, bytes, &at, st);
    if (e != hipSuccess) return e;
    const Sorted x{w.keys[at], w.poss[at], (uint32_t)s.N, (uint32_t)s.V, plan.chunk, w.head, w.tail, scale, add, s.D,
                   whole_blocks(s, grad)};
    if (s.dtype == DT_F32) return sums_t<DT_F32, DT_F32>(x, plan.chunks, g, grad, st);
    if (grad_dtype == DT_F32) return sums_t<DT_BF16, DT_F32>(x, plan.chunks, g, grad, st);
    return sums_t<DT_BF16, DT_BF16>(x, plan.chunks, g, grad, st);
}

}  // namespace lrscan
