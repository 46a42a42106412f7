// blocks.cu -- choosing pages of a long cache: bounds of every page's keys, and
// for each query the pages whose bounds allow the largest scores.
//
// sum_i q_i k_i <= sum_i max(q_i hi_i, q_i lo_i) for every key between a page's
// bounds, channel by channel.  Bounds are 8-bit whole numbers times a power of
// two, rounded outwards, and queries 8-bit whole numbers times a power of two, so
// a score is a whole number below 2^21 times a power of two: exact in fp32, in
// whatever order it is summed, and the pages chosen do not depend on the kernel.
// Queries are rounded to nearest, so a score is a bound for the rounded query, not quite
// for the query: of normal keys and queries 87 to 92 % of the pages chosen are those of
// unrounded bounds and queries (64 of 512 pages of 64, 16 of 256 pages of 32).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/tree_attn.h"
#include "cluster.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "layout.h"
#include "mma_sync.cuh"
#include "ptx.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kExpMin = -100, kExpMax = 100;

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

// The least e of [kExpMin, kExpMax] with x <= 127 * 2^e, for x >= 0 with no more
// significant bits than bf16: x = f * 2^k with 1 <= f < 2, and 127 = 1.984375 * 2^6.
__device__ __forceinline__ int exponent_for(float x) {
    const uint32_t b = __float_as_uint(x);
    const int e = static_cast<int>(b >> 23) - 127 - 6 + ((b & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);
}
// 2^e for e in [kExpMin, kExpMax].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// ---------------------------------------------------------------------------
// Bounds.  A page of one KV head is contiguous and is read in one go.  Large bf16 pages
// (16 KB and more) have a CTA of four warps each, so that few pages fill the GPU; others a
// warp each, which needs no barrier.  Bound by memory with bf16 rows, by the conversions of
// 8-bit ones, by a page's chain (its number, its rows, the join) where pages are small.
// Measured, 64 sequences with 0.26 M tokens in all and 8 heads of 128, pages of 64: bf16
// 94 us (5.6 TB/s), 8-bit 62 (4.3 TB/s; by four warps a page and in fp32 150); 8-bit in
// pages of 16 121 (512).
// ---------------------------------------------------------------------------
struct BoundsArgs {
    const void* k_pages;
    const uint8_t* k_scales;
    const int32_t* table;
    const int32_t* starts;  // nullable: 0
    const int32_t* lens;
    int8_t* bounds;
    uint8_t* exps;
    int max_pages, Hkv, P, num_pages;
    int32_t* status;
};

constexpr int kBoundsWarps = 4;
constexpr int kBoundsThreads = 32 * kBoundsWarps;

// The codes of one (page, KV head): bounds h and l of channels `ch` .. ch + N - 1 (with
// h >= l where there is any number), all of them by the threads that share `top`, the
// largest magnitude.
template <int D, int N>
__device__ __forceinline__ void store_bounds(const BoundsArgs& a, size_t at, int ch,
                                             const float (&h)[N], const float (&l)[N], int e) {
    const float inv = pow2(-e);
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int x = static_cast<int>(fminf(fmaxf(ceilf(h[i] * inv), -127.0f), 127.0f));
        const int y = static_cast<int>(fminf(fmaxf(floorf(l[i] * inv), -127.0f), 127.0f));
        hi |= (static_cast<uint32_t>(x) & 255u) << (8 * i);
        lo |= (static_cast<uint32_t>(y) & 255u) << (8 * i);
    }
    int8_t* to = a.bounds + at * 2 * D + ch;
    if (N == 4) {
        *reinterpret_cast<uint32_t*>(to) = hi;
        *reinterpret_cast<uint32_t*>(to + D) = lo;
    } else if (N == 2) {
        *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(hi);
        *reinterpret_cast<uint16_t*>(to + D) = static_cast<uint16_t>(lo);
    } else {
        to[0] = static_cast<int8_t>(hi);
        to[D] = static_cast<int8_t>(lo);
    }
}

// Infinities as the largest finite number, 0 where there is no number at all.
__device__ __forceinline__ void finite_bounds(float& h, float& l) {
    const float most = __uint_as_float(0x7f7f0000u);
    if (!(h >= l)) h = l = 0.0f;
    h = fminf(fmaxf(h, -most), most);
    l = fminf(fmaxf(l, -most), most);
}

// The pages of sequence b that are to be done, and its length; false where there are none.
__device__ __forceinline__ bool pages_of(const BoundsArgs& a, int b, int& first, int& end, int& L) {
    bool bad;
    const int start = a.starts != nullptr ? a.starts[b] : 0;
    L = clamp_seq_len(a.lens[b], a.P, a.max_pages, bad);
    if (bad || start < 0) {
        report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
        return false;
    }
    first = start / a.P;
    end = start < L ? (L + a.P - 1) / a.P : 0;
    return first < end;
}

// Larger and smaller halves of pairs of bf16 (fp16) numbers; the number, of a number and
// a NaN.
template <bool FP8>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    if (FP8)
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool FP8>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    if (FP8)
        asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool FP8>
__device__ __forceinline__ float half_of(uint32_t pair, int i) {
    if (!FP8) return __uint_as_float(i == 0 ? pair << 16 : pair & 0xffff0000u);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(i == 0 ? pair : pair >> 16)));
}

// Four warps to a page: bf16 only.
template <int D>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int LPR = D / 8;          // lanes per row
    constexpr int RW = 32 / LPR;        // rows per load of a warp
    constexpr int STEP = RW * kBoundsWarps;
    constexpr int U = 8;
    __shared__ uint32_t part[kBoundsWarps][2][D / 2];
    __shared__ float red[kBoundsWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = blockIdx.y, b = blockIdx.z;
    int from, end, L;
    if (!pages_of(a, b, from, end, L)) return;
    const int sub = lane % LPR, row0 = warp * RW + lane / LPR;
    for (int j = from + blockIdx.x; j < end; j += gridDim.x) {
        const int page = a.table[static_cast<size_t>(b) * a.max_pages + j];
        if (page < 0 || page >= a.num_pages) {
            if (tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            continue;
        }
        const int n = min(a.P, L - j * a.P);
        const size_t at = static_cast<size_t>(page) * a.Hkv + hk;
        const uint16_t* base = static_cast<const uint16_t*>(a.k_pages) + at * a.P * D + sub * 8;
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = 0xff80ff80u;
            l[i] = 0x7f807f80u;
        }
        for (int r0 = row0; r0 < n + row0; r0 += U * STEP) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r0 + u * STEP < n)
                    x[u] = ptx::ld_stream(base + static_cast<size_t>(r0 + u * STEP) * D);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r0 + u * STEP >= n) break;
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = max_pair<false>(h[i], w[i]);
                    l[i] = min_pair<false>(l[i], w[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int off = LPR; off < 32; off <<= 1) {
                h[i] = max_pair<false>(h[i], __shfl_xor_sync(kFull, h[i], off));
                l[i] = min_pair<false>(l[i], __shfl_xor_sync(kFull, l[i], off));
            }
        }
        __syncthreads();  // (the page before has been read from `part`)
        if (lane < LPR) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                part[warp][0][sub * 4 + i] = h[i];
                part[warp][1][sub * 4 + i] = l[i];
            }
        }
        __syncthreads();
        float hi[1] = {0.0f}, lo[1] = {0.0f};
        if (tid < D) {
            uint32_t x = part[0][0][tid / 2], y = part[0][1][tid / 2];
#pragma unroll
            for (int w = 1; w < kBoundsWarps; ++w) {
                x = max_pair<false>(x, part[w][0][tid / 2]);
                y = min_pair<false>(y, part[w][1][tid / 2]);
            }
            hi[0] = half_of<false>(x, tid & 1);
            lo[0] = half_of<false>(y, tid & 1);
            finite_bounds(hi[0], lo[0]);
        }
        float top = fmaxf(fabsf(hi[0]), fabsf(lo[0]));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        top = red[0];
#pragma unroll
        for (int w = 1; w < kBoundsWarps; ++w) top = fmaxf(top, red[w]);
        const int e = exponent_for(top);
        if (tid < D) store_bounds<D, 1>(a, at, tid, hi, lo, e);
        if (tid == 0) a.exps[at] = static_cast<uint8_t>(e + 127);
    }
}

// A warp to a page.  8-bit rows: with t the largest scale of the page, values are held in
// fp16 in units of 2^t, where a code times 2^(s - t) is exact down to s - t = -15.  Rows
// below that take part with 2^-15: their values, at most 448 * 2^-15 < 2^-6 then, have
// bounds' codes of -1, 0 or 1 by their sign alone as long as the codes' unit is 2^(t - 6)
// at least; where it is not (rows whose largest code is small), the page is done again
// in fp32.
template <int D, bool FP8>
__global__ void __launch_bounds__(kBoundsThreads) bounds_warp_kernel(const BoundsArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int V = FP8 ? 16 : 8;     // values of a 16-byte vector
    constexpr int LPR = D / V;          // lanes per row
    constexpr int RW = 32 / LPR;        // rows per load of the warp
    constexpr int U = 8;
    constexpr int N = D / 32;           // channels whose codes a lane writes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.y;
    int from, end, L;
    if (!pages_of(a, b, from, end, L)) return;
    const int sub = lane % LPR, group = lane / LPR;
    const int items = (end - from) * a.Hkv, step = gridDim.x * kBoundsWarps;
    const int32_t* table = a.table + static_cast<size_t>(b) * a.max_pages + from;
    int item = blockIdx.x * kBoundsWarps + warp;
    int page_next = item < items ? table[item / a.Hkv] : 0;
    for (; item < items; item += step) {
        const int j = from + item / a.Hkv, hk = item % a.Hkv;
        const int page = page_next;
        if (item + step < items) page_next = table[(item + step) / a.Hkv];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            continue;
        }
        const int n = min(a.P, L - j * a.P);
        const size_t at = static_cast<size_t>(page) * a.Hkv + hk;
        const uint8_t* base = static_cast<const uint8_t*>(a.k_pages) +
                              at * a.P * D * (FP8 ? 1 : 2) + sub * 16;
        constexpr int RB = FP8 ? D : 2 * D;
        const uint8_t* scales = FP8 ? a.k_scales + at * a.P : nullptr;
        int t = 0;  // 8-bit rows: the largest scale byte
        if (FP8) {
            for (int r = lane; r < n; r += 32) t = max(t, static_cast<int>(scales[r]));
            t = __reduce_max_sync(kFull, t);
        }
        uint32_t h[V / 2], l[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            h[i] = FP8 ? 0xfc00fc00u : 0xff80ff80u;
            l[i] = FP8 ? 0x7c007c00u : 0x7f807f80u;
        }
        for (int r0 = group; r0 < n + group; r0 += U * RW) {
            uint4 x[U];
            uint8_t s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * RW;
                if (r < n) {
                    x[u] = ptx::ld_stream(base + static_cast<size_t>(r) * RB);
                    if (FP8) s[u] = scales[r];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r0 + u * RW >= n) break;
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                if (FP8) {
                    const __half2 f = __half2half2(__ushort_as_half(static_cast<unsigned short>(
                        max(static_cast<int>(s[u]) - t, -15) + 15 > 0
                            ? (max(static_cast<int>(s[u]) - t, -14) + 15) << 10
                            : 0x0200)));  // 2^-15 is subnormal
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t y[2];
                        f16x2_of_e4m3x4(w[i], y[0], y[1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            __half2 z = __hmul2(*reinterpret_cast<__half2*>(&y[k]), f);
                            const uint32_t v = *reinterpret_cast<uint32_t*>(&z);
                            h[2 * i + k] = max_pair<FP8>(h[2 * i + k], v);
                            l[2 * i + k] = min_pair<FP8>(l[2 * i + k], v);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h[i] = max_pair<FP8>(h[i], w[i]);
                        l[i] = min_pair<FP8>(l[i], w[i]);
                    }
                }
            }
        }
        // The lanes of a row's vector share it out as they join it: half of what a lane
        // has goes to the other one at each step, N channels are left.
#pragma unroll
        for (int off = 16, m = V / 4; off >= LPR; off >>= 1, m >>= 1) {
            const bool upper = (lane & off) != 0;
#pragma unroll
            for (int i = 0; i < m; ++i) {
                const uint32_t x = __shfl_xor_sync(kFull, upper ? h[i] : h[i + m], off);
                const uint32_t y = __shfl_xor_sync(kFull, upper ? l[i] : l[i + m], off);
                h[i] = max_pair<FP8>(upper ? h[i + m] : h[i], x);
                l[i] = min_pair<FP8>(upper ? l[i + m] : l[i], y);
            }
        }
        float hi[N], lo[N];
        const float unit = FP8 ? scale_of(t) : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            hi[i] = half_of<FP8>(h[i / 2], i & 1) * unit;
            lo[i] = half_of<FP8>(l[i / 2], i & 1) * unit;
            finite_bounds(hi[i], lo[i]);
        }
        auto exponent = [&] {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) top = fmaxf(top, fmaxf(fabsf(hi[i]), fabsf(lo[i])));
            // (bits of numbers >= 0 are in the numbers' order)
            return exponent_for(__uint_as_float(
                __reduce_max_sync(kFull, __float_as_uint(top))));
        };
        int e = exponent();
        const int ch = sub * V + group * N;
        if (FP8 && e < t - 127 - 6) {  // (rare) the same in fp32
#pragma unroll
            for (int i = 0; i < N; ++i) {
                hi[i] = -INFINITY;
                lo[i] = INFINITY;
            }
            for (int r = 0; r < n; ++r) {
                const float f = scale_of(scales[r]);
                const uint8_t* row = static_cast<const uint8_t*>(a.k_pages) + (at * a.P + r) * D + ch;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float y = half_of<true>(f16x2_of_e4m3x2(row[i]), 0) * f;
                    hi[i] = fmaxf(hi[i], y);
                    lo[i] = fminf(lo[i], y);
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) finite_bounds(hi[i], lo[i]);
            e = exponent();
        }
        store_bounds<D, N>(a, at, ch, hi, lo, e);
        if (lane == 0) a.exps[at] = static_cast<uint8_t>(e + 127);
    }
}

// ---------------------------------------------------------------------------
// Selection.  A cluster of CTAs takes the pages of one (sequence, KV head) for
// some of its tokens.  With p = max(c, 0) and m = min(c, 0) a score is
// p . hi + m . lo: a product of the pages' bounds (16 pages to a tile, 2 d deep)
// with the query codes, on the tensor cores in fp16, whose products and fp32 sums
// of such whole numbers are exact.
//
// The bounds of a page are contiguous and each is used once, so they go from
// memory straight into the product's registers: the order of channels within a
// product is free, and is chosen so that a lane's 16 bytes are its operand.
//
// The k-th highest score is found by counting: the keys (ordered bits of the scores)
// between the lowest and the highest fall into 256 equal ranges, the one with the k-th
// is divided again, until it holds no more than are wanted of it; two counts as a rule.
// The pages are then written in their order.
//
// Measured, 64 sequences of 512 to 16384 tokens, 4 tokens each, 32 heads on 8 of 128, 64
// pages of 16 tokens taken: 31 us (67 MB of bounds, 2.1 TB/s).  Bound by the rate of
// instructions and their latency -- 400 to a tile of 16 pages, of which 160 widen the codes;
// a third of the time is the choice -- with three CTAs to an SM (two: 37 us, four, which
// spill: 63).  One token of 512 pages takes 6 us, latency alone.  The host lays a CTA out for
// the table's width, not for the lengths: from 3457 columns on such a CTA has two of the four
// tokens, from 7489 on one, and reads the bounds twice or four times (the same sequences:
// 32 us up to 2048 columns, 42 with 3456, 37 with 4096, 66 with 8192, 80 with 16384).
// ---------------------------------------------------------------------------
struct SelectArgs {
    const uint16_t* q;
    const int8_t* bounds;
    const uint8_t* exps;
    const int32_t* table;
    const int32_t* lens;
    int32_t* blocks;
    int max_pages, Hq, Hkv, T, P, num_pages, n_select, n_first, n_last;
    int TC, chunks;  // tokens of a CTA, and CTAs' worth of tokens
    int cols;        // columns of a token: a power of two up to 8, or a multiple of 8
    int per_most;    // scores of a token that one CTA holds at most
    bool gather;     // whether a CTA has room for all scores of a token of the cluster
    int B;
    bool longest_first;
    int32_t* status;
};

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;

// Order-preserving bits of a score (above 1, the key of a page that scores nothing).
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}

// Four int8 codes as two fp16 pairs: 1024 + (code + 128) has the byte as its last
// bits, and the difference is exact.
__device__ __forceinline__ void f16x2_of_s8x4(uint32_t x, uint32_t& h0, uint32_t& h1) {
    const uint32_t u = x ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 y0 = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
    __half2 y1 = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    h0 = *reinterpret_cast<uint32_t*>(&y0);
    h1 = *reinterpret_cast<uint32_t*>(&y1);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// The keys of one token, spread over the cluster's CTAs, `per` to each.
struct Keys {
    uint32_t at;  // of the token's scores in this CTA's shared memory
    int per;
    bool remote;
    __device__ __forceinline__ uint32_t operator()(int i) const {
        if (!remote) {
            uint32_t v;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at + 4 * i) : "memory");
            return v;
        }
        const int r = i / per;
        return ld_cluster_u32(ptx::map_rank(at + 4 * (i - r * per), r));
    }
};

// Barrier of the NW warps that work on one token: all of the CTA's, some, or one.
template <int NW>
__device__ __forceinline__ void group_sync(int id) {
    if (NW == kSelWarps)
        __syncthreads();
    else if (NW > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "n"(32 * NW) : "memory");
    else
        __syncwarp();
}

struct Scratch {  // of the warps that work on one token
    int hist[256];
    uint32_t low[kSelWarps], high[kSelWarps];
    int counts[2 * kSelWarps];
};

constexpr int kHeld = 16;  // keys that a lane may hold in registers

// By NW warps: of keys lo .. hi - 1 (none of them 0), the k highest (ties: the lowest
// indices), together with all indices of [0, lo) and [hi, n), as ascending indices to out.
// HELD: n <= 32 NW kHeld, so that each key is read once and stays in a register.
template <int NW, bool HELD>
__device__ __forceinline__ void take_highest(const Keys& key, int n, int lo, int hi, int k,
                                             int32_t* out, Scratch& sc, int id, int t) {
    constexpr int GS = 32 * NW;
    const int lane = t & 31, w = t >> 5;
    const int seg = ((n + GS - 1) / GS) * 32;  // keys of one warp, in a row
    const int a0 = min(w * seg, n), a1 = min(a0 + seg, n);
    uint32_t held[HELD ? kHeld : 1];
    auto read = [&](int i) { return i >= max(lo, a0) && i < min(hi, a1) ? key(i) : 0u; };
    if (HELD) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) held[HELD ? j : 0] = read(a0 + 32 * j + lane);
    }
    // f(index, key) for each of this lane's keys, 0 for what is not a candidate.
    auto each = [&](auto f) {
        if (HELD) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                if (a0 + 32 * j >= a1) break;
                f(a0 + 32 * j + lane, held[HELD ? j : 0]);
            }
        } else {
#pragma unroll 4
            for (int i0 = a0; i0 < a1; i0 += 32) f(i0 + lane, read(i0 + lane));
        }
    };
    uint32_t bound = 0xffffffffu;  // keys above it are taken, and the first `left` equal to it
    int left = 0;
    if (k > 0) {
        uint32_t low = 0xffffffffu, high = 0;  // (low: less one, so that 0 is the largest)
        each([&](int, uint32_t v) {
            low = min(low, v - 1u);
            high = max(high, v);
        });
        low = __reduce_min_sync(kFull, low);
        high = __reduce_max_sync(kFull, high);
        if (NW > 1) {
            if (lane == 0) {
                sc.low[w] = low;
                sc.high[w] = high;
            }
            group_sync<NW>(id);
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                low = min(low, sc.low[i]);
                high = max(high, sc.high[i]);
            }
        }
        low += 1;
        left = k;  // still to be found among keys low .. high
        for (;;) {
            const uint32_t range = high - low;
            const int shift = max(0, 24 - __clz(range));
            for (int i = t; i < 256; i += GS) sc.hist[i] = 0;
            group_sync<NW>(id);
            each([&](int, uint32_t v) {  // (0 - low is above every range)
                if (v - low <= range) atomicAdd(sc.hist + ((v - low) >> shift), 1);
            });
            group_sync<NW>(id);
            // The range that holds the left-th from the top; every warp finds it.
            // Of the 256 counts, which 32 first, then which of them.
            int eighth = 0, above = 0;
            {
                int part[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    part[j] = __reduce_add_sync(kFull, sc.hist[255 - (lane + 32 * j)]);
#pragma unroll
                for (int j = 0; j < 7; ++j) {
                    const bool on = eighth == j && above + part[j] < left;
                    above += on ? part[j] : 0;
                    eighth += on;
                }
            }
            const int mine = sc.hist[255 - (32 * eighth + lane)];
            int upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(kFull, upto, off);
                if (lane >= off) upto += y;
            }
            const int src = __ffs(__ballot_sync(kFull, above + upto >= left)) - 1;
            const int in = __shfl_sync(kFull, mine, src);
            left -= above + __shfl_sync(kFull, upto, src) - in;
            low += static_cast<uint32_t>(255 - (32 * eighth + src)) << shift;
            if (in == left || shift == 0) {  // all of the range, or keys that are all equal
                bound = low;
                break;
            }
            high = min(high, low + ((1u << shift) - 1u));
            group_sync<NW>(id);  // (hist has been read)
        }
    }
    // Keys above the bound, and the first `left` that equal it (all of those, where the
    // whole range is taken).
    auto taken = [&](int i, uint32_t v) {
        return i < a1 && (i < lo || i >= hi || v > bound);
    };
    int more = 0, same = 0;
    if (NW > 1) {
        each([&](int i, uint32_t v) {
            more += __popc(__ballot_sync(kFull, taken(i, v)));
            same += __popc(__ballot_sync(kFull, v == bound));
        });
        if (lane == 0) {
            sc.counts[2 * w] = more;
            sc.counts[2 * w + 1] = same;
        }
        group_sync<NW>(id);
        more = same = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            more += i < w ? sc.counts[2 * i] : 0;
            same += i < w ? sc.counts[2 * i + 1] : 0;
        }
    }
    const unsigned below = (1u << lane) - 1u;
    each([&](int i, uint32_t v) {
        const bool over = taken(i, v);
        const unsigned gt = __ballot_sync(kFull, over);
        const unsigned eq = __ballot_sync(kFull, v == bound);
        const int eq_rank = same + __popc(eq & below);
        if (over || (v == bound && eq_rank < left))
            out[more + __popc(gt & below) + min(eq_rank, left)] = i;
        more += __popc(gt);
        same += __popc(eq);
    });
    group_sync<NW>(id);
}

// TILES: column tiles that share one conversion of the bounds (the last of several such
// turns may work on columns that nobody wants).
template <int D, int TILES>
__global__ void __launch_bounds__(kSelThreads, 3) select_kernel(const SelectArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    // Query codes: [column][16-byte vectors of codes as (p, p, m, m) pairs], columns 64
    // bytes apart beyond their length: two rows' reads fall on different banks.
    constexpr int kStride = 4 * D + 64;  // bytes
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int S = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    const int unit = blockIdx.x / S;
    const int hk = unit / a.chunks % a.Hkv;
    int b = unit / (a.chunks * a.Hkv);
    if (a.longest_first) b = by_length(a.lens, a.B, b, reinterpret_cast<int*>(smem));
    const int t0 = unit % a.chunks * a.TC;
    const int nt = min(a.TC, a.T - t0);  // tokens
    const int G = a.Hq / a.Hkv;
    const int tiles = ((a.TC * a.cols + 7) / 8 + TILES - 1) / TILES * TILES;
    uint8_t* codes = smem;                                                // [tiles * 8][kStride]
    Scratch* scratch = reinterpret_cast<Scratch*>(codes + tiles * 8 * kStride);  // [kSelWarps]
    uint32_t* scores = reinterpret_cast<uint32_t*>(scratch + kSelWarps);  // [TC][per_most]
    // The pages' numbers stand where the first token's scores will: a warp has read those
    // of a tile, and of its next, before it writes the tile's scores.
    int* pages = reinterpret_cast<int*>(scores);

    bool bad;
    const int L = clamp_seq_len(a.lens[b], a.P, a.max_pages, bad);
    if (bad && tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    const int nb = (L + a.P - 1) / a.P;
    const int per = max((nb + S - 1) / S, 1);
    const int lo = min(rank * per, nb), hi = min(lo + per, nb);

    if (nb > a.n_select) {
        const int32_t* table = a.table + static_cast<size_t>(b) * a.max_pages;
        for (int i = lo + tid; i < hi; i += kSelThreads) pages[i - lo] = table[i];
        __syncthreads();
        constexpr int NC = D / 64;  // 16-byte vectors of a row of bounds, to a lane
        // Columns: one, two, four or eight to a token, or `wide` tiles.
        const int log_cols = 31 - __clz(min(a.cols, 8)), per_tile = 8 >> log_cols;
        const int t_lane = 2 * c >> log_cols, wide = a.cols >> 3;
        const bool writes = (2 * c & ((1 << log_cols) - 1)) == 0;
        // A tile's loads: the bounds of pages g and g + 8, their exponents.
        uint4 x[2][2][NC];  // [page g, g + 8][hi, lo]
        uint8_t exps[2];
        unsigned missing = 0;  // bits of pages that are not in the pool
        auto fetch = [&](int p0) {
            missing = 0;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                int page = pages[min(p0 + g + 8 * r, hi - 1) - lo];
                if (page < 0 || page >= a.num_pages) {
                    report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                    missing |= 1u << r;
                    page = 0;
                }
                const size_t at = static_cast<size_t>(page) * a.Hkv + hk;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < NC; ++j)
                        x[r][h][j] = ptx::ld_stream(a.bounds + at * 2 * D + h * D + j * 64 + c * 16);
                exps[r] = a.exps[at];
            }
        };
        if (lo + warp * 16 < hi) fetch(lo + warp * 16);
        // Query codes, while the first bounds are on their way: a token's heads by one warp,
        // or by `parts` of them.
        const int tokens = tiles * 8 / a.cols;
        const int parts = tokens <= 1 ? kSelWarps : tokens <= 2 ? kSelWarps / 2
                          : tokens <= kSelWarps / 2 ? 2 : 1;
        for (int t = warp / parts; t < tokens; t += kSelWarps / parts) {
            const uint16_t* q =
                a.q + ((static_cast<size_t>(b) * a.T + min(t0 + t, a.T - 1)) * a.Hq + hk * G) * D;
            uint32_t top = 0;
            for (int i = lane; i < G * D / 2; i += 32) {
                const uint32_t x = reinterpret_cast<const uint32_t*>(q)[i];
                const uint32_t l = x & 0x7fffu, h = (x >> 16) & 0x7fffu;
                top = max(top, l < 0x7f80u ? l : 0u);
                top = max(top, h < 0x7f80u ? h : 0u);
            }
            top = __reduce_max_sync(kFull, top);
            const float inv = pow2(-exponent_for(__uint_as_float(top << 16)));
            // Four codes at a time: vector j, word w of lane c is channels 64 j + 16 c + 4 w.
            for (int i = warp % parts * 32 + lane; i < a.cols * D / 4; i += 32 * parts) {
                const int col = i / (D / 4), d = i % (D / 4) * 4;
                const uint2 raw = *reinterpret_cast<const uint2*>(
                    q + (col < G ? col : 0) * D + d);  // columns past the group repeat its first
                __half2 p[2], m[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = h == 0 ? raw.x : raw.y;
                    float y[2] = {__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)};
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        y[e] = y[e] != y[e] ? 0.0f
                                            : fminf(fmaxf(rintf(y[e] * inv), -127.0f), 127.0f);
                    p[h] = __floats2half2_rn(fmaxf(y[0], 0.0f), fmaxf(y[1], 0.0f));
                    m[h] = __floats2half2_rn(fminf(y[0], 0.0f), fminf(y[1], 0.0f));
                }
                const int j = d / 64, lane_c = d / 16 % 4, w = d / 4 % 4;
                uint4 v;
                v.x = *reinterpret_cast<uint32_t*>(&p[0]);
                v.y = *reinterpret_cast<uint32_t*>(&p[1]);
                v.z = *reinterpret_cast<uint32_t*>(&m[0]);
                v.w = *reinterpret_cast<uint32_t*>(&m[1]);
                *reinterpret_cast<uint4*>(codes + (t * a.cols + col) * kStride + (j * 4 + w) * 64 +
                                          lane_c * 16) = v;
            }
        }
        __syncthreads();
        for (int p0 = lo + warp * 16; p0 < hi; p0 += kSelWarps * 16) {
            const float size[2] = {scale_of(exps[0]), scale_of(exps[1])};
            const bool none[2] = {(missing & 1u) != 0, (missing & 2u) != 0};
            __syncwarp();
            for (int n0 = 0; n0 < tiles; n0 += TILES) {
                float acc[TILES][4];
#pragma unroll
                for (int n = 0; n < TILES; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll
                for (int j = 0; j < NC; ++j) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t f[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const uint4 v = x[r][h][j];
                                f16x2_of_s8x4(w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w,
                                              f[h][r], f[h][r + 2]);
                            }
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            const uint4 q = *reinterpret_cast<const uint4*>(
                                codes + ((n0 + n) * 8 + g) * kStride + (j * 4 + w) * 64 + c * 16);
                            ptx::mma_sync_f16(acc[n], f[0][0], f[0][1], f[0][2], f[0][3], q.x, q.y);
                            ptx::mma_sync_f16(acc[n], f[1][0], f[1][1], f[1][2], f[1][3], q.z, q.w);
                        }
                    }
                }
                // The next tile's loads, once this one's bounds have been used.
                if (n0 + TILES >= tiles && p0 + kSelWarps * 16 < hi) fetch(p0 + kSelWarps * 16);
                // The largest of each token's columns.
#pragma unroll
                for (int n = 0; n < TILES; ++n) {
                    // Token of this lane's first column (of `wide` tiles, the same of all).
                    const int t = wide > 1 ? (n0 + n) / wide : (n0 + n) * per_tile + t_lane;
                    const bool again = wide > 1 && (n0 + n) % wide != 0;
                    uint32_t* to = scores + t * a.per_most + (p0 + g - lo);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float y0 = acc[n][2 * r], y1 = acc[n][2 * r + 1];
                        if (a.cols > 1) y0 = fmaxf(y0, y1);
                        if (a.cols > 2) y0 = fmaxf(y0, __shfl_xor_sync(kFull, y0, 1));
                        if (a.cols > 4) y0 = fmaxf(y0, __shfl_xor_sync(kFull, y0, 2));
                        if (!writes || p0 + g + 8 * r >= hi || t >= nt) continue;
                        uint32_t k = none[r] ? 1u : score_key(y0 * size[r]);
                        if (again) k = max(k, to[8 * r]);
                        to[8 * r] = k;
                        if (a.cols == 1 && t + 1 < nt)
                            to[a.per_most + 8 * r] = none[r] ? 1u : score_key(y1 * size[r]);
                    }
                }
            }
        }
    }
    if (S > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    // Tokens are shared out over the cluster's CTAs, and a CTA's over its warps.
    Keys key;
    key.per = per;
    key.remote = S > 1;
    auto row_of = [&](int t) {
        return a.blocks +
               ((static_cast<size_t>(b) * a.T + t0 + t) * a.Hkv + hk) * a.n_select;
    };
    const int k = min(a.n_select, nb);
    for (int t = rank; t < nt; t += S) {
        int32_t* out = row_of(t);
        for (int i = tid; i < a.n_select; i += kSelThreads)
            if (i >= k || nb == k) out[i] = i < k ? i : -1;
    }
    if (nb > a.n_select) {  // (so the first and the last ones do not meet)
        const int here = (nt - rank + S - 1) / S;  // tokens of this CTA
        auto take = [&](auto warps, auto in_registers) {
            constexpr int NW = decltype(warps)::value;
            const int group = warp / NW;
            for (int t = rank + S * group; t < nt; t += S * (kSelWarps / NW)) {
                key.at = ptx::smem_u32(scores + static_cast<size_t>(t) * a.per_most);
                if (!decltype(in_registers)::value && key.remote && a.gather) {
                    // (NW is all warps here) One round of reads from the others, not five.
                    uint32_t* all = scores + static_cast<size_t>(a.TC) * a.per_most;
#pragma unroll 8
                    for (int i = tid; i < nb; i += kSelThreads) all[i] = key(i);
                    __syncthreads();
                    Keys near = key;
                    near.remote = false;
                    near.at = ptx::smem_u32(all);
                    take_highest<NW, false>(near, nb, a.n_first, nb - a.n_last,
                                            k - a.n_first - a.n_last, row_of(t), scratch[group],
                                            group, tid);
                    continue;
                }
                take_highest<NW, decltype(in_registers)::value>(
                    key, nb, a.n_first, nb - a.n_last, k - a.n_first - a.n_last, row_of(t),
                    scratch[group], group, tid % (32 * NW));
            }
        };
        using std::integral_constant;
        constexpr int kOf = 32 * kHeld;  // keys that a warp holds
        if (here >= 8 && nb <= kOf)
            take(integral_constant<int, 1>(), std::true_type());
        else if (here >= 3 && nb <= 2 * kOf)
            take(integral_constant<int, 2>(), std::true_type());
        else if (here >= 2 && nb <= 4 * kOf)
            take(integral_constant<int, 4>(), std::true_type());
        else if (nb <= 8 * kOf)
            take(integral_constant<int, 8>(), std::true_type());
        else
            take(integral_constant<int, 8>(), std::false_type());
    }
    if (S > 1) ptx::cluster_sync();  // (other CTAs may still read this one's scores)
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

bool cache_shape_ok(int B, int Hkv, int d, int max_pages, int P, int num_pages) {
    return B >= 0 && B <= 65535 && Hkv >= 1 && Hkv <= 65535 && (d == 64 || d == 128) &&
           max_pages >= 1 && num_pages >= 1 && page_size_ok(P) &&
           static_cast<long long>(num_pages) * Hkv * P < (1LL << 31) &&
           static_cast<long long>(max_pages) * P < (1LL << 31);
}

constexpr int kMaxSelectPages = 262144;

// Column tiles of so many columns that share a conversion, and how many there are then.
int tiles_at_once(int columns) { return columns <= 8 ? 1 : columns <= 16 ? 2 : 4; }
int padded_tiles(int columns) {
    const int n = tiles_at_once(columns);
    return ((columns + 7) / 8 + n - 1) / n * n;
}

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_kv_block_bounds(const void* k_pages, const uint8_t* k_scales, const int32_t* block_table,
                         int max_pages_per_seq, const int32_t* starts, const int32_t* seq_lens,
                         int8_t* bounds, uint8_t* bounds_exp, int B, int Hkv, int d,
                         int page_size, int num_pages, int32_t* status, void* stream) {
    if (!cache_shape_ok(B, Hkv, d, max_pages_per_seq, page_size, num_pages) ||
        static_cast<long long>(max_pages_per_seq) * Hkv >= (1LL << 30))
        return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    if (!k_pages || !block_table || !seq_lens || !bounds || !bounds_exp) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(k_pages, 16) || !ptr_aligned(bounds, 16) || !ptr_aligned(block_table, 4) ||
        !ptr_aligned(starts, 4) || !ptr_aligned(seq_lens, 4) || !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    const int sms = sms_of(dev);
    if (sms == 0) return TREE_ATTN_ERR_CUDA;
    BoundsArgs a;
    a.k_pages = k_pages;
    a.k_scales = k_scales;
    a.table = block_table;
    a.starts = starts;
    a.lens = seq_lens;
    a.bounds = bounds;
    a.exps = bounds_exp;
    a.max_pages = max_pages_per_seq;
    a.Hkv = Hkv;
    a.P = page_size;
    a.num_pages = num_pages;
    a.status = status;
    // The host does not know how many pages a sequence has: its CTAs take them in turn,
    // eight to an SM where there are that many.
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k_scales == nullptr && page_size * d >= 64 * 128) {
        const long long rows = static_cast<long long>(B) * Hkv;
        const long long fill = (8LL * sms + rows - 1) / rows;
        const int nx = static_cast<int>(fill < max_pages_per_seq ? fill : max_pages_per_seq);
        return rc_of(launch_dependent(d == 128 ? bounds_kernel<128> : bounds_kernel<64>,
                                      dim3(nx, Hkv, B), dim3(kBoundsThreads), 0, s, a));
    }
    const long long fill = (8LL * sms + B - 1) / B;
    const long long most =
        (static_cast<long long>(max_pages_per_seq) * Hkv + kBoundsWarps - 1) / kBoundsWarps;
    const int nx = static_cast<int>(fill < most ? fill : most);
    using Kernel = void (*)(BoundsArgs);
    const Kernel kernel =
        k_scales ? (d == 128 ? bounds_warp_kernel<128, true> : bounds_warp_kernel<64, true>)
                 : (d == 128 ? bounds_warp_kernel<128, false> : bounds_warp_kernel<64, false>);
    return rc_of(launch_dependent(kernel, dim3(nx, B), dim3(kBoundsThreads), 0, s, a));
}

int tree_select_blocks(const uint16_t* q, const int8_t* bounds, const uint8_t* bounds_exp,
                       const int32_t* block_table, int max_pages_per_seq, const int32_t* seq_lens,
                       int32_t* blocks, int B, int Hq, int Hkv, int d, int T, int page_size,
                       int num_pages, int n_select, int n_first, int n_last, int32_t* status,
                       void* stream) {
    if (!cache_shape_ok(B, Hkv, d, max_pages_per_seq, page_size, num_pages) || T < 1 ||
        T > TREE_ATTN_MAX_T || Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > 128 || n_select < 1 ||
        n_select > 4096 || n_first < 0 || n_last < 0 || n_first > n_select - n_last ||
        max_pages_per_seq > kMaxSelectPages)
        return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    if (!q || !bounds || !bounds_exp || !block_table || !seq_lens || !blocks)
        return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(q, 16) || !ptr_aligned(bounds, 16) || !ptr_aligned(block_table, 4) ||
        !ptr_aligned(seq_lens, 4) || !ptr_aligned(blocks, 4) || !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    const int sms = sms_of(dev);
    if (sms == 0) return TREE_ATTN_ERR_CUDA;
    const int G = Hq / Hkv;
    SelectArgs a;
    a.q = q;
    a.bounds = bounds;
    a.exps = bounds_exp;
    a.table = block_table;
    a.lens = seq_lens;
    a.blocks = blocks;
    a.max_pages = max_pages_per_seq;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.T = T;
    a.P = page_size;
    a.num_pages = num_pages;
    a.n_select = n_select;
    a.n_first = n_first;
    a.n_last = n_last;
    a.status = status;
    a.cols = 1;
    while (a.cols < G && a.cols < 8) a.cols *= 2;
    if (G > 8) a.cols = (G + 7) / 8 * 8;
    // CTAs of a cluster: as many as fill the SMs twice, while each has four tiles.
    int S = 1;
    while (S < 8 && 2LL * S * B * Hkv <= 2LL * sms && max_pages_per_seq >= 2 * S * 64) S *= 2;
    // Tokens of a CTA: all, unless its scores or its query codes get too large.
    const size_t code_row = static_cast<size_t>(4 * d + 64);
    int TC = T;
    size_t need = 0;
    for (;; TC = (TC + 1) / 2) {
        a.per_most = ((max_pages_per_seq + S - 1) / S + 3) / 4 * 4;
        need = static_cast<size_t>(TC) * a.per_most * 4 + kSelWarps * sizeof(Scratch) +
               static_cast<size_t>(padded_tiles(TC * a.cols) * 8) * code_row;
        // (72 KB: three CTAs to an SM; 227 KB: all that a CTA can have, which the widest tables
        // with 97 heads and more to a group take)
        if (need <= (TC > 1 ? 72u * 1024u : S < 8 ? 200u * 1024u : 227u * 1024u)) break;
        if (TC == 1) {  // one token of a very long sequence: more CTAs share its pages
            if (S == 8) return TREE_ATTN_ERR_SHAPE;
            S *= 2;
            TC = 2;  // (1 again)
        }
    }
    a.gather = S > 1 && max_pages_per_seq > 32 * kHeld * kSelWarps &&
               need + static_cast<size_t>(max_pages_per_seq) * 4 <= 200u * 1024u;
    if (a.gather) need += static_cast<size_t>(max_pages_per_seq) * 4;
    a.TC = TC;
    a.B = B;
    a.longest_first = B > 1 && B <= kSelThreads &&
                      static_cast<long long>(B) * Hkv * ((T + TC - 1) / TC) > 2LL * sms;
    a.chunks = (T + TC - 1) / TC;
    const long long grid = static_cast<long long>(B) * Hkv * a.chunks * S;
    if (grid >= (1LL << 31)) return TREE_ATTN_ERR_SHAPE;
    using Kernel = void (*)(SelectArgs);
    const int at_once = tiles_at_once(TC * a.cols);
    const Kernel kernel =
        d == 128 ? (at_once == 1   ? select_kernel<128, 1>
                    : at_once == 2 ? select_kernel<128, 2>
                                   : select_kernel<128, 4>)
                 : (at_once == 1   ? select_kernel<64, 1>
                    : at_once == 2 ? select_kernel<64, 2>
                                   : select_kernel<64, 4>);
    static std::atomic<unsigned long long> ready[2][3];
    if (need > 48 * 1024 && !opt_in(reinterpret_cast<const void*>(kernel), dev,
                                    ready[d == 128][at_once == 4 ? 2 : at_once - 1]))
        return TREE_ATTN_ERR_CUDA;
    return rc_of(launch_cluster(kernel, dim3(static_cast<unsigned>(grid)), dim3(kSelThreads), need,
                                S, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
