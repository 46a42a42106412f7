// beam.cu -- beam search's selection: the best continuations over all beams of
// a sequence and the whole vocabulary.
//
// With x the logits of beam w and s_w its score, candidate (w, v) scores
//   s_w + (x_v - m) - ln sum_u exp(x_u - m),   m = max x,
// and the K highest are taken, ties to the lowest (w, v).  Within a beam that
// is the order of x itself, so one pass over the logits suffices: a CTA takes a
// piece of a row, keeps it in registers, and leaves the piece's maximum, its
// sum of exponentials (fp32) and its K largest logits.  A second, small kernel
// joins the sums, scores the few candidates in fp64 (so that the order of two
// beams' candidates is not that of a rounding) and takes the best K.
//
// The K largest of a piece: the largest logit of every group of four lanes is
// known after the maximum; the K-th largest of those 64 is a bound that at least
// K logits reach and few exceed, and only logits at or above it are looked at
// again.  Keys (logit, -index) are all different, so ties need no extra rule.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tree_attn.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kEach = 32;                  // logits of one thread
constexpr int kPiece = kThreads * kEach;   // logits of one CTA
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving bits of a logit (-0 as +0, NaN as -inf: no candidate).
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.0f; }
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key >> 31) != 0 ? key & 0x7fffffffu : ~key);
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
    int W, V, K, pieces;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) piece_kernel(const PieceArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ unsigned long long piece_found[];  // K * 4 * kEach at most
    __shared__ unsigned long long tops[kThreads];
    __shared__ float red[kWarps];
    __shared__ unsigned long long bound;
    __shared__ int n_found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.y, piece = blockIdx.x;
    const int b = row / a.W, w = row % a.W;
    if (a.finished != nullptr && a.finished[row] != 0) return;  // (not read for it either)
    const T* x = static_cast<const T*>(a.logits) + b * a.batch_stride + w * a.beam_stride;
    const int first = piece * kPiece;
    constexpr int N = 16 / sizeof(T);  // logits of a vector
    constexpr int U = kEach / N;
    // Vectors start on 16-byte boundaries: `skew` logits before the row's first
    // belong to the first one, and are not read.
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    float v[kEach];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = first + (u * kThreads + tid) * N - skew;
        if (i >= 0 && i + N <= a.V) {
            const uint4 raw = *reinterpret_cast<const uint4*>(x + i);
            const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
            for (int j = 0; j < N; ++j) v[u * N + j] = as_float<T>(t[j]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                v[u * N + j] = i + j >= 0 && i + j < a.V ? as_float<T>(x[i + j]) : -INFINITY;
        }
    }
    // The largest of each thread; of two equal ones the first.
    float top = -INFINITY;
    int at = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        v[e] = clean(v[e]);
        if (v[e] > top) {
            top = v[e];
            at = e;
        }
    }
    auto index_of = [&](int e) {
        return static_cast<uint32_t>(first + ((e / N) * kThreads + tid) * N - skew + e % N);
    };
    unsigned long long mine =
        top == -INFINITY
            ? 0ull
            : (static_cast<unsigned long long>(key_of(top)) << 32) | (0xffffffffu - index_of(at));
    float m = top;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    if (lane == 0) red[warp] = m;
    // Groups of four lanes where 64 tops are enough, else every lane its own.
    const int group = a.K <= 16 ? 4 : 1;
    if (group == 4) {
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            const unsigned long long o = __shfl_xor_sync(kFull, mine, off);
            mine = o > mine ? o : mine;
        }
        if ((lane & 3) == 0) tops[tid >> 2] = mine;
    } else {
        tops[tid] = mine;
    }
    if (tid == 0) {
        n_found = 0;
        bound = 1;  // any candidate, unless there are K tops
    }
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) m = fmaxf(m, red[i]);
    const int n_tops = kThreads / group;
    if (tid < n_tops) {
        const unsigned long long t = tops[tid];
        int above = 0;
#pragma unroll 8
        for (int i = 0; i < n_tops; ++i) above += tops[i] > t;
        if (t != 0 && above == a.K - 1) bound = t;
    }
    float sum = 0.0f;
    if (m == INFINITY) {  // such logits share all of the probability
#pragma unroll
        for (int e = 0; e < kEach; ++e) sum += v[e] == INFINITY ? 1.0f : 0.0f;
    } else if (m > -INFINITY) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) sum += exp2f((v[e] - m) * kLog2e);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    const unsigned long long lim = bound;
    const float least = logit_of(static_cast<uint32_t>(lim >> 32));
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (lim == 1 ? v[e] > -INFINITY : v[e] >= least) {
            const unsigned long long k = (static_cast<unsigned long long>(key_of(v[e])) << 32) |
                                         (0xffffffffu - index_of(e));
            if (k >= lim) piece_found[atomicAdd(&n_found, 1)] = k;
        }
    }
    __syncthreads();
    const int n = n_found;
    const size_t out = static_cast<size_t>(row) * a.pieces + piece;
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long k = piece_found[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += piece_found[j] > k;
        if (above < a.K) a.keys[out * a.K + above] = k;
    }
    for (int i = n + tid; i < a.K; i += kThreads) a.keys[out * a.K + i] = 0;
    if (tid == 0) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += red[i];
        a.sums[out] = make_float2(m, s);
    }
}

// ---------------------------------------------------------------------------
// Joining: one CTA per sequence.
// ---------------------------------------------------------------------------
struct JoinArgs {
    const unsigned long long* keys;
    const float2* sums;
    const float* scores;      // [B][W]
    const uint8_t* finished;  // nullable
    float* scores_out;        // [B][K]
    int32_t* rows_out;        // [B][K]
    int32_t* tokens_out;      // [B][K]
    int W, V, K, pieces, eos;
};

constexpr int kJoinThreads = 256;
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

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ Cand join_found[];  // K * (candidates per thread) at most
    __shared__ Cand tops[kJoinThreads];
    __shared__ double log_sum[kMaxBeams];
    __shared__ float row_max[kMaxBeams];
    __shared__ Cand bound;
    __shared__ int n_found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x;
    const size_t row0 = static_cast<size_t>(b) * a.W;
    for (int w = warp; w < a.W; w += kJoinThreads / 32) {
        float m = -INFINITY;
        const bool done = a.finished != nullptr && a.finished[row0 + w] != 0;
        const float2* s = a.sums + (row0 + w) * a.pieces;
        if (!done)
            for (int i = lane; i < a.pieces; i += 32) m = fmaxf(m, s[i].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        double sum = 0.0;
        if (!done && m > -INFINITY)
            for (int i = lane; i < a.pieces; i += 32)
                if (s[i].x > -INFINITY)
                    sum += s[i].x == m ? s[i].y
                                       : static_cast<double>(s[i].y) * exp2f((s[i].x - m) * kLog2e);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
        if (lane == 0) {
            row_max[w] = m;
            log_sum[w] = done ? 0.0 : log(sum);
        }
    }
    if (tid == 0) {
        n_found = 0;
        bound.s = 1;
        bound.place = 0;
    }
    __syncthreads();
    const int per_row = a.pieces * a.K;
    const int all = a.W * per_row;
    auto cand = [&](int i) {
        Cand c;
        c.s = 0;
        c.place = 0;
        const int w = i / per_row, j = i - w * per_row;
        const double start = a.scores[row0 + w];
        if (a.finished != nullptr && a.finished[row0 + w] != 0) {  // stands for itself alone
            if (j == 0) {
                c.s = bits_of(start);
                c.place = ~(static_cast<unsigned long long>(w) * a.V + a.eos);
            }
            return c;
        }
        const unsigned long long k = a.keys[(row0 + w) * per_row + j];
        if (k != 0) {
            const double x = logit_of(static_cast<uint32_t>(k >> 32));
            const double top = row_max[w];
            c.s = bits_of(start + ((x == top ? 0.0 : x - top) - log_sum[w]));
            c.place = ~(static_cast<unsigned long long>(w) * a.V +
                        (0xffffffffu - static_cast<uint32_t>(k)));
        }
        return c;
    };
    Cand mine;
    mine.s = mine.place = 0;
    for (int i = tid; i < all; i += kJoinThreads) {
        const Cand c = cand(i);
        if (better(c, mine)) mine = c;
    }
    tops[tid] = mine;
    __syncthreads();
    if (mine.s != 0) {
        int above = 0;
        for (int i = 0; i < kJoinThreads; ++i) above += better(tops[i], mine);
        if (above == a.K - 1) bound = mine;
    }
    __syncthreads();
    const Cand lim = bound;
    for (int i = tid; i < all; i += kJoinThreads) {
        const Cand c = cand(i);
        if (!better(lim, c)) join_found[atomicAdd(&n_found, 1)] = c;
    }
    __syncthreads();
    const int n = n_found;
    const size_t out = static_cast<size_t>(b) * a.K;
    for (int i = tid; i < n; i += kJoinThreads) {
        const Cand c = join_found[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += better(join_found[j], c);
        if (above < a.K) {
            const unsigned long long flat = ~c.place;
            const int w = static_cast<int>(flat / a.V);
            a.scores_out[out + above] = static_cast<float>(score_of(c.s));
            a.rows_out[out + above] = static_cast<int>(row0) + w;
            a.tokens_out[out + above] =
                static_cast<int>(flat - static_cast<unsigned long long>(w) * a.V);
        }
    }
    for (int i = n + tid; i < a.K; i += kJoinThreads) {
        a.scores_out[out + i] = -INFINITY;
        a.rows_out[out + i] = -1;
        a.tokens_out[out + i] = -1;
    }
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

// Pieces of a row: one more than V asks for, for rows that start inside a vector.
int pieces_of(int V) { return (V + 7 + kPiece - 1) / kPiece; }

bool beam_shape_ok(int B, int W, int V, int K) {
    return B >= 0 && W >= 1 && W <= kMaxBeams && V >= 1 && K >= 1 && K <= kMaxBeams &&
           V <= (1 << 30) && static_cast<long long>(B) * W <= 65535 &&
           static_cast<long long>(W) * pieces_of(V) * K <= 32768;
}

// Candidates the join may have to keep: K threads' worth of them.
size_t join_smem(int W, int V, int K) {
    const int all = W * pieces_of(V) * K;
    return static_cast<size_t>(K) * ((all + kJoinThreads - 1) / kJoinThreads) * sizeof(Cand);
}
size_t piece_smem(int K) {
    return static_cast<size_t>(K) * (K <= 16 ? 4 : 1) * kEach * sizeof(unsigned long long);
}

size_t beam_bytes(int B, int W, int V, int K) {
    const size_t n = static_cast<size_t>(B) * W * pieces_of(V);
    return (n * K * 8 + n * 8 + 255) / 256 * 256;
}

bool allow_smem(const void* kernel, size_t bytes) {
    return bytes <= 32 * 1024 ||
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(bytes)) == cudaSuccess;
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
    if (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < beam_bytes(B, W, V, K))
        return TREE_ATTN_ERR_WORKSPACE;
    const int pieces = pieces_of(V);
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
    using Kernel = void (*)(PieceArgs);
    const Kernel kernel = dtype == 2   ? piece_kernel<float>
                          : dtype == 1 ? piece_kernel<__half>
                                       : piece_kernel<__nv_bfloat16>;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!allow_smem(reinterpret_cast<const void*>(kernel), piece_smem(K)) ||
        !allow_smem(reinterpret_cast<const void*>(join_kernel), join_smem(W, V, K)))
        return TREE_ATTN_ERR_CUDA;
    const int rc = rc_of(launch_dependent(kernel, dim3(pieces, B * W), dim3(kThreads),
                                          piece_smem(K), s, p));
    if (rc != TREE_ATTN_OK) return rc;
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
    return rc_of(launch_dependent(join_kernel, dim3(B), dim3(kJoinThreads), join_smem(W, V, K), s,
                                  j));
}

}  // extern "C"
