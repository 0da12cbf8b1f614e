// conv.hip -- the short causal convolution over tokens, one filter of K taps
// for each channel, with an optional sigmoid-weighted activation:
//
//   z_t = bias + sum_j w[j] x_{t-K+1+j},     y_t = z_t  or  z_t sigmoid(z_t)
//   gz_t = g_t dy/dz,   dx_s = sum_back w[K-1-back] gz_{s+back},
//   dw[j] = sum_t gz_t x_{t-K+1+j},   dbias = sum_t gz_t
//
// Inputs before the first come from `state` (the K - 1 inputs before it) or are
// zero, and a tap that would reach across a reset counts as zero.
//
// A thread owns four adjacent channels of a chunk of consecutive
// tokens and walks it in groups of tokens whose rows are loaded together.  The
// last K - 1 inputs stay in registers, so a chunk re-reads only K - 1 rows of
// its neighbour; a reset clears them, which drops an infinity or NaN of the
// segment before.  The backward walks in the same order, recomputes z, and
// keeps the K - 1 input gradients that still wait for later gz in registers.
// The parameter gradients are summed over the chunk in registers, over a
// workgroup's chunks through LDS, and over workgroups by column_sum, each in a
// fixed order.
//
// Resets and the ends of a row are rare, so what they need runs under
// wavefront-wide branches; everything else is straight-line code, in which the
// moving window costs no instruction.  (With a test of every thread at every
// row the window was moved through copies, a quarter of all instructions.)
//
// Bound (MI355X, bf16 [8, 2048, 2560], K = 4, with resets and activation,
// caches flushed): forward 37 us for 168 MB (4.5 TB/s), the vector units busy
// for 21; reverse 68 us, 5 of them the parameters' sums, for 252 MB (3.7 TB/s),
// the vector units busy for 42: four wavefronts a SIMD, each with a group of
// rows in flight, cover neither wholly.  Smaller calls leave a SIMD two
// wavefronts (bf16 [8, 2048, 1024] 39 us for 101 MB), and rows that are not
// whole quads take twice the time ([8, 2048, 1023] 90 us).
#include "conv.hpp"

#include <type_traits>

#include "column_sum.hpp"
#include "gated_math.hpp"
#include "launch.hpp"
#include "quad.hpp"

namespace lrscan {

namespace {

constexpr int kBlock = 256;
// Tokens whose rows are loaded together: a multiple of K - 1, so that the
// window's and the waiting gradients' places in their rings are constants.
constexpr int group_of(int K) { return K == 4 ? 6 : 4; }

constexpr int V = kQuad;  // channels of a thread

// Tokens of a chunk.  The backward's walk goes K - 1 tokens past its chunk, so
// that walk is what is a whole number of groups.
//
// Long chunks re-read less, short ones make more wavefronts.  The forward takes
// two groups of tokens, three of rows that a wavefront holds several of, as
// long as that leaves six wavefronts for each of the 256 CUs, and else one: its
// wavefronts lie side by side along the rows in pairs, so that the rows in
// flight lie together.  Measured on MI355X (bf16, us, K = 4, in chunks of 6, 12,
// 18 and 48 tokens, four wavefronts side by side): [16, 4096, 2560] 148, 135, 135,
// 143; [16, 2048, 1024] 34, 32, 33, 32; [64, 2048, 128] 21, 21, 18, 25; [1, 2048,
// 1024] 7, 8, 10, 17.  Pairs take up to 10% less ([32, 1024, 1536] 45 against 50),
// single ones 6% more on long rows (142 against 134).  For the reverse see
// bwd_rows.
//
// A thread of four channels beats one of eight (reverse 72 against 85, forward
// 43 against 48, [8, 2048, 2560] bf16): its state leaves four wavefronts a SIMD in
// the reverse walk and eight in the forward one.
constexpr uint32_t kFwdWidth = 128, kBwdWidth = 64;  // threads along a row, at most
constexpr int kFwdGroups = 3, kBwdGroups = 14;       // of tokens in a walk, at most
int fwd_rows(const ConvShape& s);
int bwd_rows(const ConvShape& s);

// Workgroup blockIdx.x covers lane block blockIdx.x % ncb and `groups`
// consecutive chunks (a chunk: `rows` tokens of one batch row).
struct ConvGrid {
    uint32_t tpr;      // threads along a row (a power of two, at most kBlock)
    uint32_t groups;   // kBlock / tpr chunks side by side
    uint32_t vpr;      // quads in a row
    uint32_t ncb;      // lane blocks
    uint32_t nchunks;  // chunks of a batch row
    uint32_t chunks;   // B * nchunks
    uint32_t blocks;   // workgroups along the chunks
    int rows;
};

int64_t chunks_of(const ConvShape& s, int rows) { return s.B * ((s.T + rows - 1) / rows); }

ConvGrid conv_grid(const ConvShape& s, int rows, uint32_t widest) {
    ConvGrid g;
    g.rows = rows;
    g.vpr = (uint32_t)((s.D + V - 1) / V);
    g.tpr = 1;
    while (g.tpr < widest && g.tpr < g.vpr) g.tpr *= 2;
    g.groups = kBlock / g.tpr;
    g.ncb = (g.vpr + g.tpr - 1) / g.tpr;
    g.nchunks = (uint32_t)((s.T + rows - 1) / rows);
    g.chunks = (uint32_t)chunks_of(s, rows);
    g.blocks = (g.chunks + g.groups - 1) / g.groups;
    return g;
}

int fwd_rows(const ConvShape& s) {
    const int u = group_of(s.K);
    const int64_t per = (s.D + V * 64 - 1) / (V * 64);  // wavefronts to a row
    for (int n = s.D > 32 * V ? 2 : kFwdGroups; n > 1; --n)
        if (s.B * ((s.T + n * u - 1) / (n * u)) * per >= 1536) return n * u;
    return u;
}

// The reverse's chunks are few and long, so what counts is how they fill the
// GPU.  A CU holds four workgroups; c of them side by side take a time of about
// (c + 2) (walk + 3 tokens), and the launch that of its fullest CU.  The walk
// with the least is taken.  Measured on MI355X (us, K = 4, in walks of 24, 36,
// 48, 60 and 72 tokens; the one taken in brackets):
//   bf16 [8,2048,2560]    74    75   [69]   70    76
//        [16,4096,2560]  242   230   227   225   226  [222 in 84]
//        [8,2048,1024]    38   [38]   43    50    49
//        [16,2048,1024]   62   [58]   57    64    62
//   fp32 [4,2048,4096]    91   [86]   86    91    81
// (By the longest walk that left six wavefronts a CU: [64,2048,128] 50, now 37;
// [1,32768,1024] 64, now 56.)
int bwd_rows(const ConvShape& s) {
    const int u = group_of(s.K);
    int best = 2;
    int64_t least = 0;
    for (int n = 2; n <= kBwdGroups; ++n) {
        const ConvGrid g = conv_grid(s, n * u - (s.K - 1), kBwdWidth);
        const int64_t all = (int64_t)g.ncb * g.blocks, left = (all % 1024 + 255) / 256;
        const int64_t cost = (n * u + 3) * (all / 1024 * 6 + (left ? left + 2 : 0));
        if (n == 2 || cost < least) best = n, least = cost;
    }
    return best * u - (s.K - 1);
}

struct ConvPos {
    int64_t bi, t0, t1, d0;  // batch row, tokens [t0, t1), first channel
    int nvalid;              // channels of the quad that exist; 0: an idle thread
};

// UNI: a wavefront lies in one chunk (rows of more than 32 quads), so chunk,
// tokens and row addresses are scalars.
template <bool UNI>
__device__ __forceinline__ ConvPos conv_pos(const ConvGrid& g, int64_t T, int64_t D) {
    const uint32_t cb = blockIdx.x % g.ncb, rb = blockIdx.x / g.ncb;
    const uint32_t lane = threadIdx.x & (g.tpr - 1);
    const uint32_t grp = UNI ? uniform((int)(threadIdx.x / g.tpr)) : threadIdx.x / g.tpr;
    const uint32_t chunk = rb * g.groups + grp, vec = cb * g.tpr + lane;
    ConvPos p;
    p.nvalid = 0;
    p.bi = p.t0 = p.t1 = p.d0 = 0;
    if (chunk >= g.chunks) return p;
    const uint32_t b = chunk / g.nchunks;
    p.bi = b;
    p.t0 = (int64_t)(chunk - b * g.nchunks) * g.rows;
    p.t1 = p.t0 + g.rows < T ? p.t0 + g.rows : T;
    p.d0 = (int64_t)vec * V;
    p.nvalid = vec >= g.vpr ? 0 : (int)((D - p.d0) < V ? (D - p.d0) : V);
    return p;
}

// Whether a condition on the chunk holds for some thread of the wavefront.
template <bool UNI>
__device__ __forceinline__ bool some(bool c) {
    if constexpr (UNI) return c;
    else return __any(c);
}

template <int K>
struct Taps {
    float w[K][V], bias[V] = {0.0f, 0.0f, 0.0f, 0.0f};
    __device__ __forceinline__ static void row(const float* p, int nvalid, float (&v)[V]) {
        const Quad<DT_F32> q = Quad<DT_F32>::load<false>(reinterpret_cast<const char*>(p), nvalid);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = q.get(j);
    }
    __device__ __forceinline__ void load(const float* wp, const float* bp, const ConvPos& p, int64_t D) {
#pragma unroll
        for (int k = 0; k < K; ++k) row(wp + k * D + p.d0, p.nvalid, w[k]);
        if (bp) row(bp + p.d0, p.nvalid, bias);
    }
    // The window is a ring whose oldest token is at place `u` modulo K - 1.
    template <int DT>
    __device__ __forceinline__ float z(const Quad<DT> (&win)[K - 1], const Quad<DT>& x, int u, int j) const {
        float z = bias[j];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) z = fmaf(w[k][j], win[(u + k) % (K - 1)].get(j), z);
        return fmaf(w[K - 1][j], x.get(j), z);
    }
};

// Segment starts of a chunk whose walk has up to WALK tokens.  A wavefront in
// one chunk reads the mask of the whole walk (the window before it too) with
// one load for every 64 tokens, a token to a lane, and keeps it as scalars;
// otherwise each thread reads its group's bytes.  (With one word for walks of
// 84 tokens the starts past token 60 were lost.)
template <bool UNI, int K, int WALK>
struct Starts {
    static constexpr int kWords = (WALK + K - 1 + kWave - 1) / kWave;
    static_assert(kWords <= 2, "a group is taken from at most two words");
    const uint8_t* row;  // mask of the batch row, or NULL
    int64_t t0, T;
    unsigned long long bits[kWords];  // UNI: bit i of word w for token t0 - (K - 1) + 64 w + i
    __device__ __forceinline__ void init(const uint8_t* reset, int64_t bi, int64_t from, int64_t len) {
        row = reset ? reset + bi * len : nullptr;
        t0 = from;
        T = len;
        if constexpr (UNI) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                bits[w] = 0;
                if (reset) {
                    const int64_t t = t0 - (K - 1) + w * kWave + (int64_t)(threadIdx.x % kWave);
                    bits[w] = __ballot(t >= 0 && t < T && row[t < 0 ? 0 : (t < T ? t : T - 1)] != 0);
                }
            }
        }
    }
    __device__ __forceinline__ bool at(int64_t t) const {  // for the window
        if constexpr (UNI) return (bits[0] >> (int)(t - t0 + K - 1)) & 1u;
        else return row && t >= 0 && row[t];
    }
    // tokens t .. t + U - 1 of the walk, bit u for token t + u
    template <int U>
    __device__ __forceinline__ uint32_t group(int64_t t) const {
        if constexpr (UNI) {
            const int at = (int)(t - t0) + K - 1;  // 1 or more
            unsigned long long w = bits[0];
            if constexpr (kWords == 1) w >>= at;
            else w = at < kWave ? (w >> at) | (bits[1] << (kWave - at)) : bits[1] >> (at - kWave);
            return (uint32_t)w & ((1u << U) - 1u);
        }
        if (!row) return 0;
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < T && row[t + u]) m |= 1u << u;
        return m;
    }
};

// The K - 1 inputs before token t0, oldest first, those of an earlier segment
// cleared.
template <int DT, bool FULL, bool UNI, int K, int WALK>
__device__ __forceinline__ void conv_warm(Quad<DT> (&win)[K - 1], const Rows& x, const void* state,
                                          const Starts<UNI, K, WALK>& starts, const ConvPos& p, int64_t D,
                                          uint32_t lo) {
    constexpr int S = Elem<DT>::bytes;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t t = p.t0 - (K - 1) + j;
        if (t >= 0)
            win[j] = Quad<DT>::template load<FULL>(x.row(p.bi, t) + lo, p.nvalid);
        else if (state)
            win[j] = Quad<DT>::template load<FULL>(
                static_cast<const char*>(state) + (size_t)((p.bi * (K - 1) + t + K - 1) * D) * S + lo,
                p.nvalid);
        else
            win[j] = Quad<DT>::zero();
        if (starts.at(t)) {
#pragma unroll
            for (int i = 0; i < j; ++i) win[i] = Quad<DT>::zero();
        }
    }
}

// The rows of a group; those past token T - 1 (ANY: there may be some) are that
// token's.
template <int DT, bool FULL, bool ANY, int U>
__device__ __forceinline__ void load_group(Quad<DT> (&r)[U], const char* p, size_t st, uint32_t lo, int64_t t,
                                           int64_t T, int nvalid) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int64_t d = u;
        if (ANY && t + u >= T) d = T - 1 - t;  // may lie before the group
        r[u] = Quad<DT>::template load<FULL>(p + (ptrdiff_t)st * d + lo, nvalid);
    }
}

template <int DT, bool FULL, bool UNI, int K, bool SILU>
__global__ __launch_bounds__(kBlock) void conv_fwd_kernel(ConvFwd a, ConvGrid g, int64_t T, int64_t D) {
    constexpr int S = Elem<DT>::bytes, U = group_of(K);
    const ConvPos p = conv_pos<UNI>(g, T, D);
    const uint32_t lo = (uint32_t)p.d0 * S;  // this thread's bytes into a row
    Starts<UNI, K, kFwdGroups * U> st;
    st.init(a.reset, p.bi, p.t0, T);  // with every lane, idle ones too
    if (p.nvalid == 0) return;
    Taps<K> tp;
    tp.load(a.w, a.bias, p, D);
    Quad<DT> win[K - 1];
    conv_warm<DT, FULL, UNI, K>(win, a.x, a.state, st, p, D, lo);
    const char* px = a.x.row(p.bi, p.t0);
    const size_t so = (size_t)D * S;
    char* po = static_cast<char*>(a.out) + (size_t)(p.bi * T + p.t0) * so;
    int head = 0;  // the ring's oldest token
    for (int64_t t = p.t0; t < p.t1; t += U) {
        const uint32_t starts = st.template group<U>(t);
        Quad<DT> x[U];
        if (some<UNI>(t + U > T)) load_group<DT, FULL, true>(x, px, a.x.st, lo, t, T, p.nvalid);
        else load_group<DT, FULL, false>(x, px, a.x.st, lo, t, T, p.nvalid);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (some<UNI>(((starts >> u) & 1u) && t + u < p.t1)) {
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    if (((starts >> u) & 1u) && t + u < p.t1) win[j] = Quad<DT>::zero();
            }
            float y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float z = tp.z(win, x[u], u, j);
                y[j] = SILU ? z * sigmoid_f(z) : z;
            }
            Quad<DT> o;
            o.set(y);
            if (t + u < p.t1) {
                o.template store<FULL>(po + so * u + lo, p.nvalid);
                win[u % (K - 1)] = x[u];
                head = (u + 1) % (K - 1);
            }
        }
        px += a.x.st * U;
        po += so * U;
    }
    if (a.last && p.t1 == T) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int back = j >= head ? j - head : j - head + K - 1;  // place in the window, oldest first
            win[j].template store<FULL>(
                static_cast<char*>(a.last) + (size_t)((p.bi * (K - 1) + back) * D) * S + lo, p.nvalid);
        }
    }
}

template <int DT, bool FULL, bool UNI, int K, bool SILU>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(UNI ? 4 : 2)))
void conv_bwd_kernel(ConvBwd a, ConvGrid g, int64_t T, int64_t D, float* part) {
    constexpr int S = Elem<DT>::bytes, U = group_of(K);
    __shared__ float s_part[kBlock * V];
    const ConvPos p = conv_pos<UNI>(g, T, D);
    const uint32_t lo = (uint32_t)p.d0 * S;  // this thread's bytes into a row
    Starts<UNI, K, kBwdGroups * U> st;
    st.init(a.reset, p.bi, p.t0, T);  // with every lane, idle ones too
    float dw[K][V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        db[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][j] = 0.0f;
    }
    if (p.nvalid > 0) {
        Taps<K> tp;
        tp.load(a.w, a.bias, p, D);
        Quad<DT> win[K - 1];
        conv_warm<DT, FULL, UNI, K>(win, a.x, a.state, st, p, D, lo);
        float acc[K - 1][V];  // input gradients of tokens t - K + 1 .. t - 1, in the window's ring
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
        int age = K - 1;  // tokens back that still lie in the segment (capped)
        const size_t so = (size_t)D * S;
        const char* px = a.x.row(p.bi, p.t0);
        const char* pg = static_cast<const char*>(a.g) + (size_t)(p.bi * T + p.t0) * so;
        // of token t - K + 1, which for the first tokens is not there (nor written)
        char* pq = a.gx.row(p.bi, p.t0) - a.gx.st * (K - 1);
        const int64_t end = p.t0 + g.rows;  // one past the chunk's last token, which may lie past T
        for (int64_t t = p.t0; t < end + K - 1; t += U) {
            const uint32_t starts = st.template group<U>(t);
            Quad<DT> x[U], gr[U];
            if (some<UNI>(t + U > T)) {
                load_group<DT, FULL, true>(x, px, a.x.st, lo, t, T, p.nvalid);
                load_group<DT, FULL, true>(gr, pg, so, lo, t, T, p.nvalid);
            } else {
                load_group<DT, FULL, false>(x, px, a.x.st, lo, t, T, p.nvalid);
                load_group<DT, FULL, false>(gr, pg, so, lo, t, T, p.nvalid);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // token tu enters, and s = tu - K + 1 gets its last contribution
                const int64_t tu = t + u, s = tu - (K - 1);
                const bool start = (starts >> u) & 1u;
                if (tu < T) age = start ? 0 : (age < K - 1 ? age + 1 : K - 1);
                // tokens back whose gradient it adds to: past the last token, none
                const int reach = tu < T ? age : -1;
                if (some<UNI>(start)) {
#pragma unroll
                    for (int j = 0; j < K - 1; ++j)
                        if (start) win[j] = Quad<DT>::zero();
                }
                float gz[V], dx[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    gz[j] = gr[u].get(j);
                    if constexpr (SILU) {  // dy/dz = q (1 + z (1 - q)), q = sigmoid(z)
                        const float z = tp.z(win, x[u], u, j);
                        const float q = sigmoid_f(z);
                        gz[j] *= q * fmaf(z, 1.0f - q, 1.0f);
                    }
                }
                // the walk's last K - 1 tokens are the next chunk's, or past the last
                // one (skipped and not multiplied by 0: an infinity may be there)
                if (tu < p.t1) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        db[j] += gz[j];
                        dw[K - 1][j] = fmaf(gz[j], x[u].get(j), dw[K - 1][j]);
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) dw[k][j] = fmaf(gz[j], win[(u + k) % (K - 1)].get(j), dw[k][j]);
                    }
                }
                if (some<UNI>(reach < K - 1)) {
#pragma unroll
                    for (int i = 0; i < K - 1; ++i)
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (K - 1 - i <= reach) acc[(u + i) % (K - 1)][j] = fmaf(tp.w[i][j], gz[j], acc[(u + i) % (K - 1)][j]);
                } else {
#pragma unroll
                    for (int i = 0; i < K - 1; ++i)
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            acc[(u + i) % (K - 1)][j] = fmaf(tp.w[i][j], gz[j], acc[(u + i) % (K - 1)][j]);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dx[j] = acc[u % (K - 1)][j];
                    acc[u % (K - 1)][j] = tp.w[K - 1][j] * gz[j];
                }
                win[u % (K - 1)] = x[u];
                if (a.grad_last && s < T && T - 1 - s < K - 1 && T - 1 - s <= age) {
                    const Quad<DT> gl = Quad<DT>::template load<FULL>(
                        static_cast<const char*>(a.grad_last) +
                            (size_t)((p.bi * (K - 1) + K - 1 - (T - s)) * D) * S + lo,
                        p.nvalid);
#pragma unroll
                    for (int j = 0; j < V; ++j) dx[j] += gl.get(j);
                }
                Quad<DT> o;
                o.set(dx);
                if (s >= p.t0 && s < T && s < end)
                    o.template store<FULL>(pq + a.gx.st * u + lo, p.nvalid);
                if (a.grad_state && s < 0)  // a token of the state (p.t0 is 0)
                    o.template store<FULL>(static_cast<char*>(a.grad_state) +
                                               (size_t)((p.bi * (K - 1) + s + K - 1) * D) * S + lo,
                                           p.nvalid);
            }
            px += a.x.st * U;
            pg += so * U;
            pq += a.gx.st * U;
        }
    }
    if (!part) return;
    // the workgroup's chunks, tap by tap (the bias last)
    const uint32_t cb = blockIdx.x % g.ncb, rb = blockIdx.x / g.ncb;
    const uint32_t width = g.tpr * V;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) s_part[threadIdx.x * V + j] = k < K ? dw[k < K ? k : 0][j] : db[j];
        __syncthreads();
        for (uint32_t e = threadIdx.x; e < width; e += kBlock) {
            const int64_t d = (int64_t)cb * width + e;
            if (d < D) {
                float t = 0.0f;
                for (uint32_t q = 0; q < g.groups; ++q) t += s_part[q * width + e];
                part[((size_t)rb * (K + 1) + k) * D + d] = t;
            }
        }
    }
}

// One token: the taps' state read, used and moved on by one (a thread's own
// channels only, so the state may be updated in place).  bf16 [256, 2560],
// K = 4: 4.8 us for 10.5 MB (2.2 TB/s), one round of loads and stores long.
template <int DT, bool FULL, int K, bool SILU>
__global__ __launch_bounds__(kBlock) void conv_step_kernel(ConvFwd a, int64_t B, int64_t D, uint32_t vpr) {
    constexpr int S = Elem<DT>::bytes;
    const uint32_t vec = blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t bi = blockIdx.y;
    if (vec >= vpr) return;
    ConvPos p;
    p.bi = bi;
    p.t0 = 0;
    p.t1 = 1;
    p.d0 = (int64_t)vec * V;
    p.nvalid = (int)((D - p.d0) < V ? (D - p.d0) : V);
    const size_t lo = (size_t)p.d0 * S, so = (size_t)D * S;
    const size_t state = (size_t)bi * (K - 1) * so + lo;
    Quad<DT> win[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        win[j] = a.state ? Quad<DT>::template load<FULL>(static_cast<const char*>(a.state) + state + j * so, p.nvalid)
                         : Quad<DT>::zero();
    const Quad<DT> x = Quad<DT>::template load<FULL>(a.x.row(bi, 0) + lo, p.nvalid);
    Taps<K> tp;
    tp.load(a.w, a.bias, p, D);
    if (a.reset && a.reset[bi]) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) win[j] = Quad<DT>::zero();
    }
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float z = tp.z(win, x, 0, j);
        y[j] = SILU ? z * sigmoid_f(z) : z;
    }
    Quad<DT> o;
    o.set(y);
    o.template store<FULL>(static_cast<char*>(a.out) + (size_t)bi * so + lo, p.nvalid);
    if (a.last) {
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j)
            win[j + 1].template store<FULL>(static_cast<char*>(a.last) + state + j * so, p.nvalid);
        x.template store<FULL>(static_cast<char*>(a.last) + state + (K - 2) * so, p.nvalid);
    }
}

// Column c of the partial rows: tap c / D of channel c % D, the bias as tap K.
struct WriteParams {
    float *w, *bias;
    int64_t nw;
    __device__ __forceinline__ void put(int64_t, int64_t c, float sum) const {
        if (c < nw) {
            if (w) w[c] = sum;
        } else if (bias) {
            bias[c - nw] = sum;
        }
    }
};

template <int DT, bool FULL, bool UNI, int K>
void fwd_launch(const ConvShape& s, const ConvFwd& p, const ConvGrid& g, hipStream_t st) {
    const dim3 grid(g.ncb * g.blocks), block(kBlock);
    if (s.silu) hipLaunchKernelGGL((conv_fwd_kernel<DT, FULL, UNI, K, true>), grid, block, 0, st, p, g, s.T, s.D);
    else hipLaunchKernelGGL((conv_fwd_kernel<DT, FULL, UNI, K, false>), grid, block, 0, st, p, g, s.T, s.D);
}

template <int DT, bool FULL, bool UNI, int K>
void bwd_launch(const ConvShape& s, const ConvBwd& p, const ConvGrid& g, float* part, hipStream_t st) {
    const dim3 grid(g.ncb * g.blocks), block(kBlock);
    if (s.silu)
        hipLaunchKernelGGL((conv_bwd_kernel<DT, FULL, UNI, K, true>), grid, block, 0, st, p, g, s.T, s.D, part);
    else
        hipLaunchKernelGGL((conv_bwd_kernel<DT, FULL, UNI, K, false>), grid, block, 0, st, p, g, s.T, s.D, part);
}

template <int DT, bool FULL, bool UNI>
void fwd_taps(const ConvShape& s, const ConvFwd& p, const ConvGrid& g, hipStream_t st) {
    if (s.K == 2) fwd_launch<DT, FULL, UNI, 2>(s, p, g, st);
    else if (s.K == 3) fwd_launch<DT, FULL, UNI, 3>(s, p, g, st);
    else fwd_launch<DT, FULL, UNI, 4>(s, p, g, st);
}

template <int DT, bool FULL, bool UNI>
void bwd_taps(const ConvShape& s, const ConvBwd& p, const ConvGrid& g, float* part, hipStream_t st) {
    if (s.K == 2) bwd_launch<DT, FULL, UNI, 2>(s, p, g, part, st);
    else if (s.K == 3) bwd_launch<DT, FULL, UNI, 3>(s, p, g, part, st);
    else bwd_launch<DT, FULL, UNI, 4>(s, p, g, part, st);
}

// Wavefront-sized workgroups, to spread a small batch over the CUs.
template <int DT, bool FULL, int K>
void step_launch(const ConvShape& s, const ConvFwd& p, hipStream_t st) {
    const uint32_t vpr = (uint32_t)((s.D + V - 1) / V);
    const dim3 grid((vpr + kWave - 1) / kWave, (unsigned)s.B), block(kWave);
    if (s.silu) hipLaunchKernelGGL((conv_step_kernel<DT, FULL, K, true>), grid, block, 0, st, p, s.B, s.D, vpr);
    else hipLaunchKernelGGL((conv_step_kernel<DT, FULL, K, false>), grid, block, 0, st, p, s.B, s.D, vpr);
}

template <int DT, bool FULL>
void step_taps(const ConvShape& s, const ConvFwd& p, hipStream_t st) {
    if (s.K == 2) step_launch<DT, FULL, 2>(s, p, st);
    else if (s.K == 3) step_launch<DT, FULL, 3>(s, p, st);
    else step_launch<DT, FULL, 4>(s, p, st);
}

template <int DT>
void step_kind(const ConvShape& s, const ConvFwd& p, hipStream_t st) {
    if (s.D % V == 0) step_taps<DT, true>(s, p, st);
    else step_taps<DT, false>(s, p, st);
}

template <int DT>
void fwd_rows_kind(const ConvShape& s, const ConvFwd& p, const ConvGrid& g, hipStream_t st) {
    if (g.tpr >= kWave) s.D % V == 0 ? fwd_taps<DT, true, true>(s, p, g, st) : fwd_taps<DT, false, true>(s, p, g, st);
    else s.D % V == 0 ? fwd_taps<DT, true, false>(s, p, g, st) : fwd_taps<DT, false, false>(s, p, g, st);
}

template <int DT>
void bwd_rows_kind(const ConvShape& s, const ConvBwd& p, const ConvGrid& g, float* part, hipStream_t st) {
    if (g.tpr >= kWave)
        s.D % V == 0 ? bwd_taps<DT, true, true>(s, p, g, part, st) : bwd_taps<DT, false, true>(s, p, g, part, st);
    else
        s.D % V == 0 ? bwd_taps<DT, true, false>(s, p, g, part, st) : bwd_taps<DT, false, false>(s, p, g, part, st);
}

}  // namespace

bool conv_fits(const ConvShape& s) {
    if (s.D > ((int64_t)1 << 29)) return false;  // a row's bytes in 32 bits
    for (int dir = 0; dir < 2; ++dir) {
        const int rows = dir == 0 ? fwd_rows(s) : bwd_rows(s);
        if (chunks_of(s, rows) >= ((int64_t)1 << 31)) return false;
        const ConvGrid g = conv_grid(s, rows, dir == 0 ? kFwdWidth : kBwdWidth);
        // work-items of the grid in 32 bits
        if ((uint64_t)g.ncb * g.blocks >= ((uint64_t)1 << 32) / kBlock) return false;
    }
    return true;
}

bool conv_sums_fit(const ConvShape& s) { return column_sum_fits((s.K + 1) * s.D); }

size_t conv_part_bytes(const ConvShape& s) {
    return (size_t)conv_grid(s, bwd_rows(s), kBwdWidth).blocks * (size_t)(s.K + 1) * (size_t)s.D * 4;
}

size_t conv_sum_scratch(const ConvShape& s) {
    return column_sum_scratch(conv_grid(s, bwd_rows(s), kBwdWidth).blocks, (s.K + 1) * s.D);
}

hipError_t launch_conv_fwd(const ConvShape& s, const ConvFwd& p, hipStream_t st) {
    if (s.T == 1 && s.B <= 65535) {
        if (s.dtype == DT_F32) step_kind<DT_F32>(s, p, st);
        else step_kind<DT_BF16>(s, p, st);
        return hipGetLastError();
    }
    const ConvGrid g = conv_grid(s, fwd_rows(s), kFwdWidth);
    if (s.dtype == DT_F32) fwd_rows_kind<DT_F32>(s, p, g, st);
    else fwd_rows_kind<DT_BF16>(s, p, g, st);
    return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvShape& s, const ConvBwd& p, float* part, float* scratch,
                           float* grad_w, float* grad_bias, hipStream_t st) {
    const ConvGrid g = conv_grid(s, bwd_rows(s), kBwdWidth);
    if (s.dtype == DT_F32) bwd_rows_kind<DT_F32>(s, p, g, part, st);
    else bwd_rows_kind<DT_BF16>(s, p, g, part, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !part) return e;
    return launch_column_sum(part, (int64_t)g.blocks, (int64_t)(s.K + 1) * s.D, scratch,
                             WriteParams{grad_w, grad_bias, (int64_t)s.K * s.D}, st);
}

}  // namespace lrscan
