// beam.cu -- beam search's selection: the best continuations over all beams of
// a sequence and the whole vocabulary.
//
// With x the logits of beam w and s_w its score, candidate (w, v) scores
//   s_w + (x_v - m) - ln sum_u exp(x_u - m),   m = max x,
// and the K highest are taken, ties to the lowest (w, v).  Within a beam that
// is the order of x itself, so one pass over the logits suffices: a CTA streams a
// piece of a row and leaves the piece's maximum, its sum of exponentials (fp32)
// and its K largest logits.  A second, small kernel joins the sums, finds with error
// bounds in fp32 which candidates may be among the best K, scores those few in fp64 (so
// that no rounding but the sums' own comes into the order of two beams' candidates) and
// ranks them.  The sums' terms go by their places in the row, not by its address: beams with
// the same logits have the same sums, and tie.
//
// The K largest of a piece: of its first tile the largest logit of every group of
// four lanes is known after the maximum; the K-th largest of those 64 is a bound
// that at least K logits reach and few exceed.  Only logits above it are kept from
// then on (one comparison per tile and thread as a rule).  Where more are kept than
// there is room for -- logits that ascend or are all equal, a first tile of -inf -- the
// piece is read again with the bound of all its threads' largest logits, under which
// there is always room, keys (logit, -index) being all different.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tree_attn.h"
#include "cluster.cuh"
#include "launch.cuh"
#include "mma_sync.cuh"
#include "ptx.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kEach = 16;                  // logits of one thread in a tile
constexpr int kTile = kThreads * kEach;
constexpr int kMostTiles = 16;             // of a piece
constexpr float kLog2e = 1.4426950408889634f;

// Bytes of what the pieces of a sequence leave to be joined.
__host__ __device__ constexpr int whole_bytes(int pieces, int K) {
    return (pieces * (K * 8 + 8) + 15) / 16 * 16;
}

// Order-preserving bits of a logit (-0 as +0, NaN as -inf: no candidate).
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.0f; }
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key >> 31) != 0 ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ float as_float(T x);
template <>
__device__ __forceinline__ float as_float(float x) {
    return x;
}
template <>
__device__ __forceinline__ float as_float(__half x) {
    return __half2float(x);
}
template <>
__device__ __forceinline__ float as_float(__nv_bfloat16 x) {
    return __bfloat162float(x);
}

struct PieceArgs {
    const void* logits;
    long long batch_stride, beam_stride;  // elements
    const uint8_t* finished;              // nullable [B][W]
    unsigned long long* keys;             // [rows][pieces][K]
    float2* sums;                         // [rows][pieces] (max, sum)
    int W, V, K, pieces, tiles, room;
};

// Sorting key of a logit: 0 for what is no candidate.
__device__ __forceinline__ unsigned long long full_key(float x, uint32_t index) {
    return x == -INFINITY
               ? 0ull
               : (static_cast<unsigned long long>(key_of(x)) << 32) | (0xffffffffu - index);
}

// The K-th largest of the CTA's keys (0: none), one to a thread, 1 where there are fewer;
// to be called by all threads.
__device__ __forceinline__ unsigned long long find_bound(unsigned long long mine, int K,
                                                         unsigned long long* tops,
                                                         unsigned long long* bound) {
    const int tid = threadIdx.x;
    tops[tid] = mine;
    if (tid == 0) *bound = 1;
    __syncthreads();
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < kThreads; ++i) above += tops[i] > mine;
    if (mine != 0 && above == K - 1) *bound = mine;
    __syncthreads();
    return *bound;
}

// The K-th largest of the largest numbers of the CTA's groups of four threads (K <= 64), by
// all threads; -inf where fewer groups have any.
__device__ __forceinline__ float group_bound(float top, int K, float* tops, uint32_t* bound) {
    const int tid = threadIdx.x;
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
    if (tid % 4 == 0) tops[tid / 4] = top;
    if (tid == 0) *bound = 0xffffffffu;
    __syncthreads();
    // (each thread of a group looks at a quarter of the others)
    int above = 0;
    const float4* quarter = reinterpret_cast<const float4*>(tops) + tid % 4 * (kThreads / 64);
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) {
        const float4 t = quarter[i];
        above += (t.x > top) + (t.y > top) + (t.z > top) + (t.w > top);
    }
    above += __shfl_xor_sync(kFull, above, 1);
    above += __shfl_xor_sync(kFull, above, 2);
    if (tid % 4 == 0 && above < K) atomicMin(bound, key_of(top + 0.0f));
    __syncthreads();
    return logit_of(*bound);
}

// A row of logits.  Which thread takes a logit, and when, goes by its index in the row
// alone, so that rows of the same logits have the same sums, bit for bit, wherever they
// begin.  A row that begins inside a 16-byte vector (SKEWED: it may) is read by whole
// vectors all the same, a lane's and the next one's making up what is the lane's.
template <typename T, bool SKEWED>
struct Row {
    const T* x;
    int V, skew;  // `skew` logits before the row's first share its first vector
    static constexpr int N = 16 / sizeof(T);
    static constexpr int kVecs = kEach / N;

    // What a thread asks for of a tile: its vectors; lane 0 also the one behind its warp's.
    struct Raw {
        uint4 own[kVecs];
        uint4 behind;
    };

    // Index of logit e of a thread in the tile that begins at `first`.
    __device__ __forceinline__ int index(int first, int e) const {
        return first + static_cast<int>(threadIdx.x >> 5) * (32 * kEach) + (e / N) * (32 * N) +
               static_cast<int>(threadIdx.x & 31) * N + e % N;
    }
    // Whether a tile's vectors lie inside the row, so that they can be read whole.
    __device__ __forceinline__ bool inside(int first) const {
        if (!SKEWED || skew == 0) return first + kTile <= V;
        return first >= skew && first + kTile + N - skew <= V;
    }
    __device__ __forceinline__ void fetch(int first, Raw& raw) const {
        const T* from = SKEWED ? x - skew : x;
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
            raw.own[u] = ptx::ld_stream(from + index(first, u * N));  // (volatile: asked for here)
        if (SKEWED && skew != 0 && (threadIdx.x & 31) == 0)
            raw.behind = ptx::ld_stream(from + index(first, 0) + 32 * kEach);
    }
    static __device__ __forceinline__ uint32_t word(const uint4& v, int i) {
        return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    }
    // The logits of a thread's vectors, WORDS (and a half: HALF) of them from the next lane's.
    template <int WORDS, bool HALF>
    __device__ __forceinline__ void unpack_as(const Raw& raw, float (&v)[kEach]) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = word(raw.own[u], i);
                if (i < WORDS + HALF) {
                    // (behind lane 31's vector lies lane 0's of the next turn, or what is
                    // behind the warp's)
                    const uint32_t after =
                        word(u + 1 < kVecs ? raw.own[(u + 1) % kVecs] : raw.behind, i);
                    w[i + 4] = __shfl_sync(kFull, lane == 0 ? after : w[i], (lane + 1) & 31);
                }
            }
            uint32_t mine[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mine[i] = HALF ? __funnelshift_r(w[i + WORDS], w[i + WORDS + 1], 16) : w[i + WORDS];
            const T* t = reinterpret_cast<const T*>(mine);
#pragma unroll
            for (int j = 0; j < N; ++j) v[u * N + j] = as_float<T>(t[j]);
        }
    }
    __device__ __forceinline__ void unpack(const Raw& raw, float (&v)[kEach]) const {
        if (!SKEWED) return unpack_as<0, false>(raw, v);
        constexpr bool H = sizeof(T) == 2;
        switch (skew * static_cast<int>(sizeof(T)) / 2) {  // (the same for all of the CTA)
            case 0: return unpack_as<0, false>(raw, v);
            case 1: return unpack_as<0, H>(raw, v);
            case 2: return unpack_as<1, false>(raw, v);
            case 3: return unpack_as<1, H>(raw, v);
            case 4: return unpack_as<2, false>(raw, v);
            case 5: return unpack_as<2, H>(raw, v);
            case 6: return unpack_as<3, false>(raw, v);
            default: return unpack_as<3, H>(raw, v);
        }
    }
    // Any tile; -inf for what is not in the row.
    __device__ __forceinline__ void load(int first, float (&v)[kEach]) const {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = index(first, e);
            v[e] = i < V ? as_float<T>(x[i]) : -INFINITY;
        }
    }
    // The largest of a thread's logits; of equal ones the first.
    __device__ __forceinline__ unsigned long long largest(int first, const float (&v)[kEach]) const {
        float top = -INFINITY;
        int at = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            if (v[e] > top) {
                top = v[e];
                at = e;
            }
        }
        return full_key(clean(top), static_cast<uint32_t>(index(first, at)));
    }
};

// Sum of exp(v - m) with m >= every v; no number where m log2(e) overflows.
__device__ __forceinline__ float exp_sum(const float (&v)[kEach], float m) {
    // 2^(v log2(e) - r), r being m log2(e) rounded, and what the rounding took.
    const float r = m * kLog2e;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < kEach; ++e) s[e & 3] += ex2(fmaf(v[e], kLog2e, -r));
    return ((s[0] + s[1]) + (s[2] + s[3])) * ex2(fmaf(-m, kLog2e, r));
}

// One piece of one row, by a CTA, what is found going to keys [K] and sums once ready() has
// returned; kept: room for `a.room` keys in shared memory.
template <typename T, bool SKEWED, typename Ready>
__device__ __forceinline__ void take_piece(const PieceArgs& a, int row, int piece,
                                           unsigned long long* kept, unsigned long long* keys,
                                           float2* sums, Ready ready) {
    __shared__ __align__(16) unsigned long long tops[kThreads];  // (read by vectors of four floats)
    __shared__ float red[2][kWarps];
    __shared__ unsigned long long bound;
    __shared__ uint32_t group_least;
    __shared__ int n_kept;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = row / a.W, w = row % a.W;
    Row<T, SKEWED> r;
    r.x = static_cast<const T*>(a.logits) + b * a.batch_stride + w * a.beam_stride;
    r.V = a.V;
    r.skew = SKEWED ? static_cast<int>((reinterpret_cast<uintptr_t>(r.x) & 15) / sizeof(T)) : 0;
    const int first = piece * a.tiles * kTile;
    if (tid == 0) n_kept = 0;
    // Keeps those of a thread's logits that exceed `above` (and reach `least`).
    auto keep = [&](const float (&v)[kEach], int at, float above, unsigned long long least) {
        unsigned which = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (v[e] > above) which |= 1u << e;
        while (which != 0) {
            const int e = __ffs(which) - 1;
            which &= which - 1;
            float y[kEach / 2];  // v[e], by halves
#pragma unroll
            for (int i = 0; i < kEach / 2; ++i) y[i] = (e & 1) != 0 ? v[2 * i + 1] : v[2 * i];
#pragma unroll
            for (int i = 0; i < kEach / 4; ++i) y[i] = (e & 2) != 0 ? y[2 * i + 1] : y[2 * i];
#pragma unroll
            for (int i = 0; i < kEach / 8; ++i) y[i] = (e & 4) != 0 ? y[2 * i + 1] : y[2 * i];
            const unsigned long long k = full_key(clean((e & 8) != 0 ? y[1] : y[0]),
                                                  static_cast<uint32_t>(r.index(at, e)));
            if (k >= least) {
                const int place = atomicAdd(&n_kept, 1);
                if (place < a.room) kept[place] = k;
            }
        }
    };
    float m = -INFINITY, s = 0.0f, lim = INFINITY;
    typename Row<T, SKEWED>::Raw raw;
    if (r.inside(first)) r.fetch(first, raw);
    for (int t = 0; t < a.tiles; ++t) {
        const int at = first + t * kTile;
        if (at >= a.V) break;
        float v[kEach];
        if (r.inside(at))
            r.unpack(raw, v);
        else
            r.load(at, v);
        // The next tile is on its way while this one is looked at.
        if (t + 1 < a.tiles && r.inside(at + kTile)) r.fetch(at + kTile, raw);
        float top = -INFINITY;  // (the number, of a number and a NaN)
#pragma unroll
        for (int e = 0; e < kEach; ++e) top = fmaxf(top, v[e]);
        if (t == 0) {
            lim = group_bound(top, a.K, reinterpret_cast<float*>(tops), &group_least);
            // (the bound itself is kept: a number below it, finite where the bound is +inf, and
            // the rest by the keys)
            const float near = fminf(lim, 3.0e38f);
            if (top >= lim)
                keep(v, at, lim == -INFINITY ? lim : near - fabsf(near) * 1e-6f - 1e-30f,
                     static_cast<unsigned long long>(key_of(lim)) << 32);
        } else if (top > lim) {  // (an equal one further on is worse than K others)
            keep(v, at, lim, 1);
        }
        // What has been kept by then gives a better bound, twice.
        if ((t == 1 || t == 3) && t + 1 < a.tiles) {
            __syncthreads();
            const int n = n_kept;
            if (n >= a.K && n <= min(kThreads, a.room)) {
                const unsigned long long mine = tid < n ? kept[tid] : 0;
                int above = 0;
                if (tid < n)
                    for (int i = 0; i < n; ++i) above += kept[i] > mine;
                if (tid < n && above == a.K - 1) bound = mine;
                __syncthreads();
                lim = logit_of(static_cast<uint32_t>(bound >> 32));
            }
            __syncthreads();  // (nothing is kept before all have the bound)
        }
        if (top > m) {
            s = m == -INFINITY ? 0.0f : s * ex2((m - top) * kLog2e);
            m = top;
        }
        if (m > -INFINITY) {
            float sum = exp_sum(v, m);
            if (!(sum < INFINITY)) {  // NaN among them, or +inf: such share all of the probability
                sum = 0.0f;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const float y = clean(v[e]);
                    sum += y == m ? 1.0f : m == INFINITY ? 0.0f : ex2((y - m) * kLog2e);
                }
            }
            s += sum;
        }
    }
    // The piece's maximum and sum.
    float all = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) all = fmaxf(all, __shfl_xor_sync(kFull, all, off));
    if (lane == 0) red[0][warp] = all;
    __syncthreads();
    all = red[0][0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) all = fmaxf(all, red[0][i]);
    s = m == all ? s : m == -INFINITY || all == INFINITY ? 0.0f : s * ex2((m - all) * kLog2e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
    if (lane == 0) red[1][warp] = s;
    __syncthreads();
    ready();
    if (tid == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += red[1][i];
        *sums = make_float2(all, sum);
    }
    int n = n_kept;
    if (n > a.room) {  // (rare) the piece again
        unsigned long long mine = 0;
        for (int t = 0; t < a.tiles; ++t) {
            float v[kEach];
            r.load(first + t * kTile, v);
            const unsigned long long k = r.largest(first + t * kTile, v);
            mine = k > mine ? k : mine;
        }
        const unsigned long long least = find_bound(mine, a.K, tops, &bound);
        if (tid == 0) n_kept = 0;
        __syncthreads();
        for (int t = 0; t < a.tiles; ++t) {
            float v[kEach];
            r.load(first + t * kTile, v);
            keep(v, first + t * kTile, -INFINITY, least);
        }
        __syncthreads();
        n = n_kept;
    }
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long k = kept[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += kept[j] > k;
        if (above < a.K) keys[above] = k;
    }
    for (int i = n + tid; i < a.K; i += kThreads) keys[i] = 0;
}

template <typename T, bool SKEWED>
__global__ void __launch_bounds__(kThreads, 4) piece_kernel(const PieceArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    const int row = blockIdx.y, piece = blockIdx.x;
    if (a.finished != nullptr && a.finished[row] != 0) return;  // (not read for it either)
    const size_t out = static_cast<size_t>(row) * a.pieces + piece;
    take_piece<T, SKEWED>(a, row, piece, reinterpret_cast<unsigned long long*>(smem), a.keys + out * a.K,
                          a.sums + out, [] {});
}

// ---------------------------------------------------------------------------
// Joining: one CTA per sequence, of a kernel of its own, or (few pieces) of the cluster that
// took them.
// ---------------------------------------------------------------------------
struct JoinArgs {
    const unsigned long long* keys;
    const float2* sums;
    const float* scores;      // [B][W]
    const uint8_t* finished;  // nullable
    float* scores_out;        // [B][K]
    int32_t* rows_out;        // [B][K]
    int32_t* tokens_out;      // [B][K]
    int W, V, K, pieces, eos, group, room;
};

constexpr int kMaxBeams = 64;

// A candidate: order-preserving bits of its fp64 score (0: none), then the
// complement of (beam, token), so that larger is better.
struct Cand {
    unsigned long long s, place;
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
    return a.s > b.s || (a.s == b.s && a.place > b.place);
}
__device__ __forceinline__ unsigned long long bits_of(double x) {
    if (!(x > -INFINITY)) return 0;  // NaN and -inf are no candidates
    const unsigned long long b =
        static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
    return (b >> 63) != 0 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double score_of(unsigned long long b) {
    return __longlong_as_double(
        static_cast<long long>((b >> 63) != 0 ? b & ~(1ull << 63) : ~b));
}

// ln x for x in [1, 2^126) to 2^-24 absolute: the power of two apart, its logarithm in
// fp64.  (fp32 would hold ln 128000 to 2^-21 only, and fp64 throughout is slow.)
__device__ __forceinline__ double log_of(float x) {
    const int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
    const float f = __uint_as_float((__float_as_uint(x) & 0x7fffffu) | 0x3f800000u);  // [1, 2)
    return static_cast<double>(e) * 0.693147180559945309 + static_cast<double>(logf(f));
}

// How many of n candidates are better than each of them: n_of(i) is told for
// candidate i by one thread, where as many threads as there are for each share it.
template <int NT, typename F>
__device__ __forceinline__ void rank_all(const Cand* c, int n, F n_of) {
    const int tid = threadIdx.x;
    int P = 1;  // threads to a candidate
    while (P < 32 && 2 * P * n <= NT) P *= 2;
    for (int i0 = 0; i0 < n; i0 += NT / P) {
        const int i = i0 + tid / P;
        const Cand mine = c[min(i, n - 1)];
        int above = 0;
#pragma unroll 4
        for (int j = tid % P; j < n; j += P) above += better(c[j], mine);
        for (int off = 1; off < P; off <<= 1) above += __shfl_xor_sync(kFull, above, off);
        if (i < n && tid % P == 0) n_of(i, mine, above);
    }
}

// Sequence b by NT threads from its pieces' keys [W][pieces][K] and sums [W][pieces]; kept_of:
// room for `a.room` candidates in shared memory.
template <int NT>
__device__ __forceinline__ void join_pieces(const JoinArgs& a, int b,
                                            const unsigned long long* keys, const float2* sums,
                                            Cand* kept_of) {
    __shared__ Cand tops[NT];
    __shared__ double less[kMaxBeams];    // what is taken off a beam's logits, after its maximum
    __shared__ float row_max[kMaxBeams], start[kMaxBeams];
    __shared__ uint8_t done[kMaxBeams];
    __shared__ Cand bound;
    __shared__ uint32_t least_bound;
    __shared__ int n_kept;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = b * a.W;
    const int per_row = a.pieces * a.K;
    const int all = a.W * per_row;
    // The first few candidates of a thread stay with it; their loads come first.
    constexpr int kHeld = 4;
    unsigned long long key[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) key[h] = tid + h * NT < all ? keys[tid + h * NT] : 0ull;
    for (int w = warp; w < a.W; w += NT / 32) {
        const bool over = a.finished != nullptr && a.finished[row0 + w] != 0;
        const float2* s = sums + w * a.pieces;
        float m = -INFINITY, sum = 0.0f;
        for (int i = lane; i < a.pieces; i += 32) {
            const float2 y = s[i];
            if (over || y.x == -INFINITY) continue;
            if (y.x > m) {
                sum = m == -INFINITY ? 0.0f : sum * ex2((m - y.x) * kLog2e);
                m = y.x;
            }
            sum += y.x == m ? y.y : y.y * ex2((y.x - m) * kLog2e);
        }
        float top = m;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        sum = m == top ? sum : m == -INFINITY ? 0.0f : sum * ex2((m - top) * kLog2e);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
        if (lane == 0) {
            row_max[w] = top;
            start[w] = a.scores[row0 + w];
            done[w] = over;
            less[w] = over || top == -INFINITY ? 0.0 : log_of(sum);
        }
    }
    if (tid == 0) n_kept = 0;
    __syncthreads();
    const float per_inv = 1.0f / static_cast<float>(per_row);
    auto cand = [&](int i, unsigned long long k) {
        Cand c;
        c.s = 0;
        c.place = 0;
        // Exact: (i + 1/2) / per_row lies 1 / (2 per_row) >= W 2^-18 from a whole number
        // (131072 candidates at most), and its error is below W 2^-22.
        const int w = min(static_cast<int>((static_cast<float>(i) + 0.5f) * per_inv), a.W - 1);
        if (done[w]) {  // stands for itself alone
            if (i == w * per_row) {
                c.s = bits_of(start[w]);
                c.place = ~(static_cast<unsigned long long>(w) * a.V + a.eos);
            }
        } else if (k != 0) {
            const float x = logit_of(static_cast<uint32_t>(k >> 32)), top = row_max[w];
            const double y = x == top ? 0.0 : static_cast<double>(x) - static_cast<double>(top);
            c.s = bits_of(static_cast<double>(start[w]) + (y - less[w]));
            c.place = ~(static_cast<unsigned long long>(w) * a.V +
                        (0xffffffffu - static_cast<uint32_t>(k)));
        }
        return c;
    };
    const size_t out = static_cast<size_t>(b) * a.K;
    auto put = [&](int, const Cand& c, int above) {
        if (above >= a.K) return;
        const unsigned long long flat = ~c.place;
        const int w = static_cast<int>(flat / a.V);
        a.scores_out[out + above] = static_cast<float>(score_of(c.s));
        a.rows_out[out + above] = row0 + w;
        a.tokens_out[out + above] =
            static_cast<int>(flat - static_cast<unsigned long long>(w) * a.V);
    };
    // What a score is at least and at most, by fp32 (in units of 2^8, which leaves room
    // for numbers of any size): three sums, and start and less rounded once each.
    auto about = [&](int i, unsigned long long k, float& least, float& most) {
        const int w = min(static_cast<int>((static_cast<float>(i) + 0.5f) * per_inv), a.W - 1);
        const float from = start[w] * 0.00390625f;
        float y = 0.0f, off = 0.0f;
        bool some = k != 0;
        if (done[w]) {
            some = i == w * per_row;
        } else if (some) {
            const float x = logit_of(static_cast<uint32_t>(k >> 32)), top = row_max[w];
            y = x == top ? 0.0f : x * 0.00390625f - top * 0.00390625f;
            off = static_cast<float>(less[w]) * 0.00390625f;
        }
        const float s = from + (y - off);
        const float e = (fabsf(from) + fabsf(y) + fabsf(off)) * 4.8e-7f + 1e-37f;  // > 2^-22 of each
        some &= s > -INFINITY;
        least = some ? s - e : -INFINITY;
        most = some ? s + e : -INFINITY;
    };
    // Candidates that may be among the K best, their scores in fp64.
    bool slow = false;
    if (all <= 64) {
        if (tid < all) {
            const Cand c = cand(tid, key[0]);
            if (c.s != 0) kept_of[atomicAdd(&n_kept, 1)] = c;
        }
    } else {
        // The K-th largest of what the best of groups of four threads are at least is a bound.
        float best = -INFINITY, top[kHeld];
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            float least;
            top[h] = -INFINITY;
            if (tid + h * NT < all) {
                about(tid + h * NT, key[h], least, top[h]);
                best = fmaxf(best, least);
            }
        }
        for (int i = tid + kHeld * NT; i < all; i += NT) {
            float least, most;
            about(i, keys[i], least, most);
            best = fmaxf(best, least);
        }
        best = fmaxf(best, __shfl_xor_sync(kFull, best, 1));
        best = fmaxf(best, __shfl_xor_sync(kFull, best, 2));
        float* bests = reinterpret_cast<float*>(tops);
        if (tid % 4 == 0) bests[tid / 4] = best;
        if (tid == 0) least_bound = 0xffffffffu;
        __syncthreads();
        int above = 0;
#pragma unroll 8
        for (int i = tid % 4; i < NT / 4; i += 4) above += bests[i] > best;
        above += __shfl_xor_sync(kFull, above, 1);
        above += __shfl_xor_sync(kFull, above, 2);
        if (tid % 4 == 0 && above < a.K) atomicMin(&least_bound, key_of(best + 0.0f));
        __syncthreads();
        const float lim = logit_of(least_bound);  // (-inf where fewer groups have any)
        auto keep = [&](int i, unsigned long long k) {
            const Cand c = cand(i, k);
            if (c.s == 0) return;
            const int at = atomicAdd(&n_kept, 1);
            if (at < a.room) kept_of[at] = c;
        };
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (top[h] >= lim && top[h] > -INFINITY) keep(tid + h * NT, key[h]);
        for (int i = tid + kHeld * NT; i < all; i += NT) {
            const unsigned long long k = keys[i];
            float least, most;
            about(i, k, least, most);
            if (most >= lim && most > -INFINITY) keep(i, k);
        }
        __syncthreads();
        slow = n_kept > a.room;
    }
    if (slow) {  // (rare: many scores that fp32 does not tell apart) all of it in fp64
        __syncthreads();
        Cand mine;
        mine.s = mine.place = 0;
        for (int i = tid; i < all; i += NT) {
            const Cand c = cand(i, keys[i]);
            if (better(c, mine)) mine = c;
        }
        int n_tops = NT;
        if (a.group == 4) {
            n_tops = NT / 4;
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                Cand o;
                o.s = __shfl_xor_sync(kFull, mine.s, off);
                o.place = __shfl_xor_sync(kFull, mine.place, off);
                if (better(o, mine)) mine = o;
            }
            if (lane % 4 == 0) tops[tid / 4] = mine;
        } else {
            tops[tid] = mine;
        }
        if (tid == 0) {
            bound.s = 1;
            bound.place = 0;
            n_kept = 0;
        }
        __syncthreads();
        rank_all<NT>(tops, n_tops, [&](int, const Cand& c, int above) {
            if (c.s != 0 && above == a.K - 1) bound = c;
        });
        __syncthreads();
        const Cand lim = bound;
        for (int i = tid; i < all; i += NT) {
            const Cand c = cand(i, keys[i]);
            if (c.s != 0 && !better(lim, c)) kept_of[atomicAdd(&n_kept, 1)] = c;
        }
    }
    __syncthreads();
    const int n = n_kept;
    rank_all<NT>(kept_of, n, put);
    for (int i = n + tid; i < a.K; i += NT) {
        a.scores_out[out + i] = -INFINITY;
        a.rows_out[out + i] = -1;
        a.tokens_out[out + i] = -1;
    }
}

template <int NT>
__global__ void __launch_bounds__(NT) join_kernel(const JoinArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    const size_t row0 = static_cast<size_t>(blockIdx.x) * a.W;
    join_pieces<NT>(a, blockIdx.x, a.keys + row0 * a.pieces * a.K, a.sums + row0 * a.pieces,
                    reinterpret_cast<Cand*>(smem));
}

// A sequence whose pieces are few, by one cluster: they leave what they find in the shared
// memory of its first CTA, which joins them.  (A cluster's size is a power of two: CTAs
// past the pieces have none.)
template <typename T, bool SKEWED>
__global__ void __launch_bounds__(kThreads, 4)
    whole_kernel(const PieceArgs a, const JoinArgs j) {
    ptx::cluster_arrive();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    const int size = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    const int b = blockIdx.x / size;
    const int found = a.W * a.pieces * a.K;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(smem);
    float2* sums = reinterpret_cast<float2*>(keys + found);
    uint8_t* room = smem + whole_bytes(a.W * a.pieces, a.K);
    const int row = b * a.W + rank / a.pieces;
    const bool has = rank < a.W * a.pieces && (a.finished == nullptr || a.finished[row] == 0);
    if (has)
        take_piece<T, SKEWED>(a, row, rank % a.pieces, reinterpret_cast<unsigned long long*>(room),
                              ptx::map_generic(keys + rank * a.K, 0),
                              ptx::map_generic(sums + rank, 0),
                              [] { ptx::cluster_wait(); });  // (the first CTA is there)
    else
        ptx::cluster_wait();
    ptx::cluster_sync();
    if (rank == 0) join_pieces<kThreads>(j, b, keys, sums, reinterpret_cast<Cand*>(room));
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

// Tiles of a row.
int tiles_of(int V) { return (V + kTile - 1) / kTile; }

// Logits a piece keeps: those of K threads, where it comes to that.
int piece_room(int K, int tiles) {
    const int n = K * kEach * tiles;
    return n < 512 ? 512 : n;
}

// Tiles of a piece: those that take the least time when the SMs take the pieces in waves
// of four to an SM, a piece taking as long as its tiles and two more (measured, a warp's
// instructions: about 200 to a tile and 264 to a piece; 256 rows of 50256 logits in bf16: 13
// pieces of one tile 22 us, two of seven 15).  Both types are bound by the rate of
// instructions (two a clock of an SM) and the wait for loads, DRAM at 59 % in fp32.  Pieces
// of fp32 end at eight tiles, of which more then fit between the last where finished beams
// leave gaps: 512 rows of 128000, a fifth of them finished, 47 us with eight and 50
// with sixteen (none finished: 56 and 53).
int piece_tiles(long long rows, int V, int K, int sms, bool fp32) {
    const int all = tiles_of(V), most = fp32 ? kMostTiles / 2 : kMostTiles;
    int best = 1;
    long long least = -1;
    for (int t = 1; t <= most && t <= all; ++t) {
        if (t > 1 && piece_room(K, t) * sizeof(unsigned long long) > 48 * 1024) break;
        const long long ctas = rows * ((all + t - 1) / t);
        const long long cost = (ctas + 4LL * sms - 1) / (4LL * sms) * (t + 2);
        if (least < 0 || cost < least) {
            least = cost;
            best = t;
        }
    }
    return best;
}

// Tiles of a piece where a sequence's pieces go to one cluster, 0 where they do not: where
// sixteen CTAs make pieces of at most two tiles, and the clusters of all sequences run at
// once.  That takes the GPU as long as two kernels do (4 beams of 32000: 6.2 us), but the
// host less, and no workspace; with pieces of four tiles it would take longer (8 beams
// of 32000: 8.4 us for 6.3).
constexpr int kMostCluster = 16, kWholeTiles = 2, kMostWhole = 16;
int whole_tiles(int B, int W, int V) {
    if (W > kMostCluster || B > kMostWhole) return 0;
    const int all = tiles_of(V), pieces = kMostCluster / W;
    const int t = (all + pieces - 1) / pieces;
    return t <= kWholeTiles ? t : 0;
}

bool beam_shape_ok(int B, int W, int V, int K) {
    return B >= 0 && W >= 1 && W <= kMaxBeams && V >= 1 && K >= 1 && K <= kMaxBeams &&
           V <= (1 << 30) && static_cast<long long>(B) * W <= 65535 &&
           static_cast<long long>(W) * tiles_of(V) * K <= 131072;
}

// Threads of the join (for one sequence with 832 candidates 256 threads are 2 us faster than
// 1024, for 32 with 1024 candidates, 32 taken, 7 us slower, for one with 8192 14 us slower:
// four candidates stay with a thread, the others are read again).
int join_threads(int all) { return all < 1024 ? 256 : 1024; }

// Threads of a group, of n, whose best candidate counts: four, unless K groups' candidates
// would not fit.
int join_group(int all, int K, int n) {
    return static_cast<size_t>(K) * ((all + n - 1) / n) * 4 * sizeof(Cand) <= 128 * 1024 ? 4 : 1;
}

// Candidates the join may have to keep: all where they are few, else K groups'.
int join_room(int all, int K, int n) {
    const int most = K * ((all + n - 1) / n) * join_group(all, K, n);
    return all <= 64 ? all : most < 256 ? 256 : most;
}
// (For pieces of one tile, the most that there can be, whatever the device.)
size_t beam_bytes(int B, int W, int V, int K) {
    if (whole_tiles(B, W, V) > 0) return 0;
    const size_t n = static_cast<size_t>(B) * W * tiles_of(V);
    return (n * K * 8 + n * 8 + 255) / 256 * 256;
}

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" {

size_t tree_beam_workspace_size(int B, int W, int V, int K) {
    return beam_shape_ok(B, W, V, K) ? beam_bytes(B, W, V, K) : 0;
}

int tree_beam_select(const void* logits, int dtype, long long batch_stride, long long beam_stride,
                     const float* scores, const uint8_t* finished, int eos, float* scores_out,
                     int32_t* rows_out, int32_t* tokens_out, int B, int W, int V, int K,
                     void* workspace, size_t workspace_bytes, void* stream) {
    if (!beam_shape_ok(B, W, V, K) || dtype < 0 || dtype > 2 || batch_stride < 0 ||
        beam_stride < 0 || (finished != nullptr && (eos < 0 || eos >= V)))
        return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    if (!logits || !scores || !scores_out || !rows_out || !tokens_out) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(logits, dtype == 2 ? 4 : 2) || !ptr_aligned(scores, 4) ||
        !ptr_aligned(scores_out, 4) || !ptr_aligned(rows_out, 4) || !ptr_aligned(tokens_out, 4))
        return TREE_ATTN_ERR_ALIGN;
    const size_t need = beam_bytes(B, W, V, K);
    if (need > 0 && (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < need))
        return TREE_ATTN_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    const int sms = sms_of(dev);
    if (sms == 0) return TREE_ATTN_ERR_CUDA;
    const int whole = whole_tiles(B, W, V);
    const int tiles = whole > 0 ? whole
                                : piece_tiles(static_cast<long long>(B) * W, V, K, sms, dtype == 2);
    const int pieces = (tiles_of(V) + tiles - 1) / tiles;
    const size_t smem = static_cast<size_t>(piece_room(K, tiles)) * sizeof(unsigned long long);
    PieceArgs p;
    p.logits = logits;
    p.batch_stride = batch_stride;
    p.beam_stride = beam_stride;
    p.finished = finished;
    p.keys = static_cast<unsigned long long*>(workspace);
    p.sums = reinterpret_cast<float2*>(p.keys + static_cast<size_t>(B) * W * pieces * K);
    p.W = W;
    p.V = V;
    p.K = K;
    p.pieces = pieces;
    p.tiles = tiles;
    p.room = piece_room(K, tiles);
    JoinArgs j;
    j.keys = p.keys;
    j.sums = p.sums;
    j.scores = scores;
    j.finished = finished;
    j.scores_out = scores_out;
    j.rows_out = rows_out;
    j.tokens_out = tokens_out;
    j.W = W;
    j.V = V;
    j.K = K;
    j.pieces = pieces;
    j.eos = eos;
    const int all = W * pieces * K;
    const int threads = whole > 0 ? kThreads : join_threads(all);
    j.group = join_group(all, K, threads);
    j.room = join_room(all, K, threads);
    const size_t join_bytes = static_cast<size_t>(j.room) * sizeof(Cand);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Whether some row may begin inside a vector.
    const size_t size = dtype == 2 ? 4 : 2;
    const bool skewed = !ptr_aligned(logits, 16) || batch_stride * size % 16 != 0 ||
                        beam_stride * size % 16 != 0;
    static std::atomic<unsigned long long> piece_ready[2][3], join_ready[2], whole_ready[2][3];
    if (whole > 0) {
        using Kernel = void (*)(PieceArgs, JoinArgs);
        static const Kernel of[2][3] = {
            {whole_kernel<__nv_bfloat16, false>, whole_kernel<__half, false>,
             whole_kernel<float, false>},
            {whole_kernel<__nv_bfloat16, true>, whole_kernel<__half, true>,
             whole_kernel<float, true>}};
        const Kernel kernel = of[skewed][dtype];
        if (!opt_in(reinterpret_cast<const void*>(kernel), dev, whole_ready[skewed][dtype], true))
            return TREE_ATTN_ERR_CUDA;
        int ctas = 1;
        while (ctas < W * pieces) ctas *= 2;
        return rc_of(launch_cluster(
            kernel, dim3(static_cast<unsigned>(B) * ctas), dim3(kThreads),
            whole_bytes(W * pieces, K) + (smem > join_bytes ? smem : join_bytes), ctas, s, p, j));
    }
    using Kernel = void (*)(PieceArgs);
    static const Kernel of[2][3] = {
        {piece_kernel<__nv_bfloat16, false>, piece_kernel<__half, false>,
         piece_kernel<float, false>},
        {piece_kernel<__nv_bfloat16, true>, piece_kernel<__half, true>, piece_kernel<float, true>}};
    const Kernel kernel = of[skewed][dtype];
    using Join = void (*)(JoinArgs);
    const Join join = threads == 256 ? join_kernel<256> : join_kernel<1024>;
    if ((smem > 32 * 1024 && !opt_in(reinterpret_cast<const void*>(kernel), dev,
                                  piece_ready[skewed][dtype])) ||
        (join_bytes > 24 * 1024 &&
         !opt_in(reinterpret_cast<const void*>(join), dev, join_ready[threads != 256])))
        return TREE_ATTN_ERR_CUDA;
    const int rc = rc_of(launch_dependent(kernel, dim3(pieces, B * W), dim3(kThreads),
                                          smem, s, p));
    if (rc != TREE_ATTN_OK) return rc;
    return rc_of(launch_dependent(join, dim3(B), dim3(threads), join_bytes, s, j));
}

}  // extern "C"
