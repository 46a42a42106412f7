// fp8_cache.cu -- writing K/V rows into the paged 8-bit cache (prompt or step
// tokens packed one sequence after the other, or the accepted path of a draft
// tree) and reading them back as bf16.  The row format is fp8.cuh's.
//
// All three kernels move rows: 2d bytes of bf16 on one side, d codes and one
// scale byte on the other.  They are bound by memory traffic for prompts and
// by launch latency for single steps.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tree_attn.h"
#include "fp8.cuh"
#include "launch.cuh"
#include "layout.h"
#include "ptx.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

// Where the rows of a paged cache live.
struct Cache {
    uint8_t* pages[2];   // K, V codes [num_pages][Hkv][P][d]
    uint8_t* scales[2];  // K, V scale bytes [num_pages][Hkv][P]
    const int32_t* block_table;
    int max_pages, Hkv, P, num_pages;
    int32_t* status;
};

// One of a pair by a run-time choice (indexing a kernel argument's array by it
// would copy the arguments to local memory).
template <typename T>
__device__ __forceinline__ T pick(T const (&v)[2], int w) {
    return w == 0 ? v[0] : v[1];
}

// Row index (page, head 0, slot) of logical position pos of sequence b, in
// rows of the pools; -1, with the status set, where there is no valid page.
// Head h's row is h * P further on.
__device__ __forceinline__ long long cache_row(const Cache& c, int b, long long pos) {
    const int shift = __ffs(c.P) - 1;
    const long long slot = pos >> shift;
    if (pos < 0 || slot >= c.max_pages) {
        report(c.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
        return -1;
    }
    const int page = c.block_table[static_cast<size_t>(b) * c.max_pages + slot];
    if (page < 0 || page >= c.num_pages) {
        report(c.status, TREE_ATTN_STATUS_BAD_PAGE);
        return -1;
    }
    return static_cast<long long>(page) * c.Hkv * c.P + (pos & (c.P - 1));
}

// Whether sequence b's packed range is in order and inside [0, N].
__device__ __forceinline__ bool range_ok(const int32_t* cu, int b, int N) {
    return cu[b] >= 0 && cu[b + 1] >= cu[b] && cu[b + 1] <= N;
}

// A sequence with a sound range that holds packed token i, or -1.  The search
// by halves misses only tokens of no sequence and, where the entries do not
// ascend, some of the sound ranges: those are looked for one by one.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int N, int i) {
    int lo = 0, hi = B;  // first b in [0, B) with cu[b + 1] > i
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    auto holds = [&](int b) { return range_ok(cu, b, N) && cu[b] <= i && i < cu[b + 1]; };
    if (lo < B && holds(lo)) return lo;
    for (int b = 0; b < B; ++b)
        if (holds(b)) return b;
    return -1;
}

// Larger halves of two pairs of 16-bit numbers.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Magnitude bits of a bf16 pair; a half that is no finite number becomes 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    const uint32_t v = w & 0x7fff7fffu;
    return v & __vcmpltu2(v, 0x7f807f80u);
}

// Largest of a row's magnitude bits, held by the D/8 lanes of its group.
template <int D>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
#pragma unroll
    for (int off = D / 16; off > 0; off >>= 1) m = max2(m, __shfl_xor_sync(kFull, m, off));
    return max(m & 0xffffu, m >> 16);
}

// Eight bf16 values (one 16-byte vector) times f to eight codes.
__device__ __forceinline__ uint2 encode8(const uint4& x, float f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = e4m3x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One row by a group of D/8 lanes, 8 values to a lane: x -> codes at
// pages + row*D, scale byte at scales + row.
template <int D>
__device__ __forceinline__ void store_row(uint8_t* pages, uint8_t* scales, long long row,
                                          const uint4& x, int gl) {
    const uint32_t k = 0x7fff7fffu;
    uint32_t top = group_max<D>(max2(max2(x.x & k, x.y & k), max2(x.z & k, x.w & k)));
    // (rare) infinities and NaN do not count
    if (__any_sync(kFull, top >= 0x7f80u))
        top = group_max<D>(
            max2(max2(finite2(x.x), finite2(x.y)), max2(finite2(x.z), finite2(x.w))));
    const int byte = scale_byte(top);
    if (row < 0) return;
    *reinterpret_cast<uint2*>(pages + row * D + gl * 8) = encode8(x, inv_scale_of(byte));
    if (gl == 0) scales[row] = static_cast<uint8_t>(byte);
}

// ---------------------------------------------------------------------------
// Append: token i of the packed rows goes to position seq_lens[b] + (i - cu[b]).
// A CTA takes a few consecutive tokens: their cache rows are looked up once,
// then groups of D/8 lanes take (tensor, head, token) rows in turn, the tokens
// of one head next to one another.
// ---------------------------------------------------------------------------
struct AppendArgs {
    Cache c;
    const int32_t* seq_lens;
    const int32_t* cu;
    const uint16_t* src[2];
    long long ts[2], hs[2];  // token and head strides of k and v (elements)
    int32_t* seq_lens_out;
    int B, N;
};

// Tokens of a CTA: 16 where that fills the GPU, else 8, so that a short prompt's
// rows are spread over more of it (measured, 8192 tokens x 8 heads: append 17.8
// and 14.8 us, read 16.3 and 13.6 us; 0.26 M tokens: 247 and 308 us, 81 and 86 us
// for 0.08 M tokens read).
constexpr int kTileMost = 16, kTileLeast = 8;

template <int D, int kTile>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ long long rows[kTile];
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * kTile;
    if (tid < kTile) {
        const int i = t0 + tid;
        long long row = -1;
        if (i < a.N) {
            const int b = sequence_of(a.cu, a.B, a.N, i);
            if (b >= 0) {
                const int32_t L = a.seq_lens[b];
                if (L < 0)
                    report(a.c.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
                else
                    row = cache_row(a.c, b, static_cast<long long>(L) + (i - a.cu[b]));
            }
        }
        rows[tid] = row;
    }
    // New lengths and the check of the ranges, by the first CTA.
    if (blockIdx.x == 0) {
        for (int b = tid; b < a.B; b += kThreads) {
            const bool ok = range_ok(a.cu, b, a.N) && a.seq_lens[b] >= 0;
            if (!ok) report(a.c.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
            if (a.seq_lens_out != nullptr)
                a.seq_lens_out[b] = a.seq_lens[b] + (ok ? a.cu[b + 1] - a.cu[b] : 0);
        }
    }
    __syncthreads();
    // A group of lanes keeps its token and goes through the (tensor, head) pairs,
    // U of them at a time: their loads are all in flight before the first is used,
    // with no branch between them (a row that goes nowhere is read all the same,
    // from a token that exists).
    if (a.N == 0) return;
    constexpr int LPR = D / 8;                      // lanes per row
    constexpr int STEP = kThreads / (LPR * kTile);  // pairs per pass of the CTA
    constexpr int U = 4;
    const int gl = tid % LPR, t = tid / LPR % kTile;
    const long long row0 = rows[t];
    const int tok = min(t0 + t, a.N - 1);
    const uint16_t* src0 = a.src[0] + tok * a.ts[0] + gl * 8;
    const uint16_t* src1 = a.src[1] + tok * a.ts[1] + gl * 8;
    const int pairs = 2 * a.c.Hkv;
    for (int q0 = tid / (LPR * kTile); q0 < pairs; q0 += U * STEP) {
        uint4 x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int q = min(q0 + i * STEP, pairs - 1);
            const uint16_t* p = q < a.c.Hkv ? src0 + q * a.hs[0] : src1 + (q - a.c.Hkv) * a.hs[1];
            x[i] = *reinterpret_cast<const uint4*>(p);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int q = q0 + i * STEP;
            const int w = q < a.c.Hkv ? 0 : 1;
            const long long row = row0 < 0 || q >= pairs
                                      ? -1
                                      : row0 + static_cast<long long>(q - w * a.c.Hkv) * a.c.P;
            store_row<D>(pick(a.c.pages, w), pick(a.c.scales, w), row, x[i], gl);
        }
    }
}

// ---------------------------------------------------------------------------
// Commit: path node k of sequence b (k < accept_len[b]) goes from the tree
// buffers [B][T][Hkv][d] to position seq_lens[b] + k.  One CTA per (sequence,
// KV head).
// ---------------------------------------------------------------------------
struct CommitFp8Args {
    Cache c;
    const int32_t* seq_lens;
    const uint16_t* src[2];
    const int32_t* accept_path;
    const int32_t* accept_len;
    int32_t* seq_lens_out;
    int T;
};

template <int D>
__global__ void __launch_bounds__(kThreads) commit_kernel(const CommitFp8Args a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int tid = threadIdx.x;
    const int b = blockIdx.x, hk = blockIdx.y;
    int n = a.accept_len[b];
    const int32_t L_in = a.seq_lens[b];
    bool bad;
    const int L = clamp_seq_len(L_in, a.c.P, a.c.max_pages, bad);
    if (n < 0 || n > a.T) {
        if (tid == 0 && hk == 0) report(a.c.status, TREE_ATTN_STATUS_BAD_PATH);
        n = 0;
    }
    if (bad) {
        if (tid == 0 && hk == 0) report(a.c.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
        n = 0;
    }
    constexpr int LPR = D / 8;
    const int gl = tid % LPR;
    for (int r0 = 0; r0 < 2 * n; r0 += kThreads / LPR) {
        const int r = r0 + tid / LPR;
        const int w = r & 1, k = r >> 1;
        long long row = -1;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (k < n) {
            const int j = a.accept_path[static_cast<size_t>(b) * a.T + k];
            if (j < 0 || j >= a.T) {
                report(a.c.status, TREE_ATTN_STATUS_BAD_PATH);
            } else {
                row = cache_row(a.c, b, static_cast<long long>(L) + k);
                if (row >= 0) {
                    row += static_cast<long long>(hk) * a.c.P;
                    x = *reinterpret_cast<const uint4*>(
                        pick(a.src, w) +
                        ((static_cast<long long>(b) * a.T + j) * a.c.Hkv + hk) * D + gl * 8);
                }
            }
        }
        store_row<D>(pick(a.c.pages, w), pick(a.c.scales, w), row, x, gl);
    }
    if (hk == 0 && tid == 0 && a.seq_lens_out != nullptr) a.seq_lens_out[b] = bad ? L_in : L + n;
}

// ---------------------------------------------------------------------------
// Read: token i of the packed output is position starts[b] + (i - cu[b]) of
// sequence b, as c * 2^s in bf16 (exact: a code has four significant bits).
// ---------------------------------------------------------------------------
struct ReadArgs {
    Cache c;
    const int32_t* starts;  // nullable: 0
    const int32_t* cu;
    uint16_t* dst[2];
    int B, N;
};

// Two codes times f (a power of two) as a bf16 pair.
__device__ __forceinline__ uint32_t decode2(uint32_t codes, float f) {
    const uint32_t h = f16x2_of_e4m3x2(codes);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const uint32_t lo = __float_as_uint(v.x * f), hi = __float_as_uint(v.y * f);
    return (lo >> 16) | (hi & 0xffff0000u);
}

template <int D, int kTile>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ long long rows[kTile];
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * kTile;
    if (tid < kTile) {
        const int i = t0 + tid;
        long long row = -1;
        if (i < a.N) {
            const int b = sequence_of(a.cu, a.B, a.N, i);
            if (b >= 0) {
                const int32_t s = a.starts != nullptr ? a.starts[b] : 0;
                row = cache_row(a.c, b, s < 0 ? -1 : static_cast<long long>(s) + (i - a.cu[b]));
            }
        }
        rows[tid] = row;
    }
    if (blockIdx.x == 0)
        for (int b = tid; b < a.B; b += kThreads)
            if (!range_ok(a.cu, b, a.N)) report(a.c.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    __syncthreads();
    // As in append_kernel, 16 codes to a lane.
    constexpr int LPR = D / 16;
    constexpr int STEP = kThreads / (LPR * kTile);
    constexpr int U = 4;
    const int gl = tid % LPR, t = tid / LPR % kTile;
    const long long row0 = rows[t];
    if (row0 < 0) return;
    const int pairs = 2 * a.c.Hkv;
    const long long out0 = static_cast<long long>(t0 + t) * a.c.Hkv * D + gl * 16;
    for (int q0 = tid / (LPR * kTile); q0 < pairs; q0 += U * STEP) {
        uint4 c[U];
        uint8_t s[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int q = min(q0 + i * STEP, pairs - 1);
            const int w = q < a.c.Hkv ? 0 : 1;
            const long long row = row0 + static_cast<long long>(q - w * a.c.Hkv) * a.c.P;
            c[i] = *reinterpret_cast<const uint4*>(pick(a.c.pages, w) + row * D + gl * 16);
            s[i] = pick(a.c.scales, w)[row];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int q = q0 + i * STEP;
            if (q >= pairs) break;
            const int w = q < a.c.Hkv ? 0 : 1;
            const float f = scale_of(s[i]);
            uint4* dst = reinterpret_cast<uint4*>(
                pick(a.dst, w) + out0 + static_cast<long long>(q - w * a.c.Hkv) * D);
            dst[0] = make_uint4(decode2(c[i].x, f), decode2(c[i].x >> 16, f), decode2(c[i].y, f),
                                decode2(c[i].y >> 16, f));
            dst[1] = make_uint4(decode2(c[i].z, f), decode2(c[i].z >> 16, f), decode2(c[i].w, f),
                                decode2(c[i].w >> 16, f));
        }
    }
}

// Checks of the pools shared by the three entries.
int check_cache(const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_scales,
                const uint8_t* v_scales, const int32_t* block_table, int32_t* status) {
    if (!k_pages || !v_pages || !k_scales || !v_scales || !block_table) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(k_pages, 16) || !ptr_aligned(v_pages, 16) || !ptr_aligned(k_scales, 16) ||
        !ptr_aligned(v_scales, 16) || !ptr_aligned(block_table, 4) || !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    return TREE_ATTN_OK;
}

bool cache_shape_ok(int B, int Hkv, int d, int max_pages, int P, int num_pages) {
    return B >= 0 && Hkv >= 1 && Hkv <= 65535 && (d == 64 || d == 128) && max_pages >= 1 &&
           num_pages >= 1 && page_size_ok(P) &&
           static_cast<long long>(num_pages) * Hkv * P < (1LL << 31);
}

Cache make_cache(const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_scales,
                 const uint8_t* v_scales, const int32_t* block_table, int max_pages, int Hkv,
                 int P, int num_pages, int32_t* status) {
    Cache c;
    c.pages[0] = const_cast<uint8_t*>(k_pages);
    c.pages[1] = const_cast<uint8_t*>(v_pages);
    c.scales[0] = const_cast<uint8_t*>(k_scales);
    c.scales[1] = const_cast<uint8_t*>(v_scales);
    c.block_table = block_table;
    c.max_pages = max_pages;
    c.Hkv = Hkv;
    c.P = P;
    c.num_pages = num_pages;
    c.status = status;
    return c;
}

// Whether tiles of kTileMost tokens give every SM four CTAs.
bool fills_gpu(int N) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return true;
    return N / kTileMost >= 4 * sms;
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_kv_append_fp8(uint8_t* k_pages, uint8_t* v_pages, uint8_t* k_scales, uint8_t* v_scales,
                       const int32_t* block_table, int max_pages_per_seq,
                       const int32_t* seq_lens, const int32_t* cu_seqlens, const uint16_t* k,
                       const uint16_t* v, long long k_token_stride, long long k_head_stride,
                       long long v_token_stride, long long v_head_stride, int32_t* seq_lens_out,
                       int B, int N, int Hkv, int d, int page_size, int num_pages,
                       int32_t* status, void* stream) {
    if (!cache_shape_ok(B, Hkv, d, max_pages_per_seq, page_size, num_pages) || N < 0)
        return TREE_ATTN_ERR_SHAPE;
    if (seq_lens_out != nullptr && seq_lens_out == seq_lens) return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    const int rc = check_cache(k_pages, v_pages, k_scales, v_scales, block_table, status);
    if (rc != TREE_ATTN_OK) return rc;
    if (!seq_lens || !cu_seqlens || (N > 0 && (!k || !v))) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(seq_lens, 4) || !ptr_aligned(cu_seqlens, 4) ||
        !ptr_aligned(seq_lens_out, 4) || !ptr_aligned(k, 16) || !ptr_aligned(v, 16) ||
        k_token_stride % 8 != 0 || k_head_stride % 8 != 0 || v_token_stride % 8 != 0 ||
        v_head_stride % 8 != 0)
        return TREE_ATTN_ERR_ALIGN;
    AppendArgs a;
    a.c = make_cache(k_pages, v_pages, k_scales, v_scales, block_table, max_pages_per_seq, Hkv,
                     page_size, num_pages, status);
    a.seq_lens = seq_lens;
    a.cu = cu_seqlens;
    a.src[0] = k;
    a.src[1] = v;
    a.ts[0] = k_token_stride;
    a.ts[1] = v_token_stride;
    a.hs[0] = k_head_stride;
    a.hs[1] = v_head_stride;
    a.seq_lens_out = seq_lens_out;
    a.B = B;
    a.N = N;
    // One CTA at least: it writes the new lengths and checks the ranges.
    const bool full = fills_gpu(N);
    const int tile = full ? kTileMost : kTileLeast;
    const dim3 grid(N > 0 ? (N + tile - 1) / tile : 1);
    using Kernel = void (*)(AppendArgs);
    const Kernel kernel =
        d == 128 ? (full ? append_kernel<128, kTileMost> : append_kernel<128, kTileLeast>)
                 : (full ? append_kernel<64, kTileMost> : append_kernel<64, kTileLeast>);
    return rc_of(launch_dependent(kernel, grid, dim3(kThreads), 0,
                                  static_cast<cudaStream_t>(stream), a));
}

int tree_kv_commit_fp8(uint8_t* k_pages, uint8_t* v_pages, uint8_t* k_scales, uint8_t* v_scales,
                       const int32_t* block_table, int max_pages_per_seq,
                       const int32_t* seq_lens, const int32_t* accept_path,
                       const int32_t* accept_len, const uint16_t* tree_k, const uint16_t* tree_v,
                       int32_t* seq_lens_out, int B, int Hkv, int d, int T, int page_size,
                       int num_pages, int32_t* status, void* stream) {
    if (!cache_shape_ok(B, Hkv, d, max_pages_per_seq, page_size, num_pages) || T < 1 ||
        T > TREE_ATTN_MAX_T)
        return TREE_ATTN_ERR_SHAPE;
    if (seq_lens_out != nullptr && seq_lens_out == seq_lens) return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    const int rc = check_cache(k_pages, v_pages, k_scales, v_scales, block_table, status);
    if (rc != TREE_ATTN_OK) return rc;
    if (!seq_lens || !accept_path || !accept_len || !tree_k || !tree_v) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(seq_lens, 4) || !ptr_aligned(accept_path, 4) ||
        !ptr_aligned(accept_len, 4) || !ptr_aligned(seq_lens_out, 4) ||
        !ptr_aligned(tree_k, 16) || !ptr_aligned(tree_v, 16))
        return TREE_ATTN_ERR_ALIGN;
    CommitFp8Args a;
    a.c = make_cache(k_pages, v_pages, k_scales, v_scales, block_table, max_pages_per_seq, Hkv,
                     page_size, num_pages, status);
    a.seq_lens = seq_lens;
    a.src[0] = tree_k;
    a.src[1] = tree_v;
    a.accept_path = accept_path;
    a.accept_len = accept_len;
    a.seq_lens_out = seq_lens_out;
    a.T = T;
    return rc_of(launch_dependent(d == 128 ? commit_kernel<128> : commit_kernel<64>,
                                  dim3(B, Hkv), dim3(kThreads), 0,
                                  static_cast<cudaStream_t>(stream), a));
}

int tree_kv_read_fp8(const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_scales,
                     const uint8_t* v_scales, const int32_t* block_table, int max_pages_per_seq,
                     const int32_t* starts, const int32_t* cu_seqlens, uint16_t* k_out,
                     uint16_t* v_out, int B, int N, int Hkv, int d, int page_size, int num_pages,
                     int32_t* status, void* stream) {
    if (!cache_shape_ok(B, Hkv, d, max_pages_per_seq, page_size, num_pages) || N < 0)
        return TREE_ATTN_ERR_SHAPE;
    if (B == 0 || N == 0) return TREE_ATTN_OK;
    const int rc = check_cache(k_pages, v_pages, k_scales, v_scales, block_table, status);
    if (rc != TREE_ATTN_OK) return rc;
    if (!cu_seqlens || !k_out || !v_out) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(starts, 4) || !ptr_aligned(cu_seqlens, 4) || !ptr_aligned(k_out, 16) ||
        !ptr_aligned(v_out, 16))
        return TREE_ATTN_ERR_ALIGN;
    ReadArgs a;
    a.c = make_cache(k_pages, v_pages, k_scales, v_scales, block_table, max_pages_per_seq, Hkv,
                     page_size, num_pages, status);
    a.starts = starts;
    a.cu = cu_seqlens;
    a.dst[0] = k_out;
    a.dst[1] = v_out;
    a.B = B;
    a.N = N;
    const bool full = fills_gpu(N);
    const int tile = full ? kTileMost : kTileLeast;
    using Kernel = void (*)(ReadArgs);
    const Kernel kernel =
        d == 128 ? (full ? read_kernel<128, kTileMost> : read_kernel<128, kTileLeast>)
                 : (full ? read_kernel<64, kTileMost> : read_kernel<64, kTileLeast>);
    return rc_of(launch_dependent(kernel, dim3((N + tile - 1) / tile), dim3(kThreads), 0,
                                  static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
