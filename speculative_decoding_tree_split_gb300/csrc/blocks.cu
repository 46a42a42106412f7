// blocks.cu -- choosing pages of a long cache: bounds of every page's keys, and
// for each query the pages whose bounds allow the largest scores.
//
// sum_i q_i k_i <= sum_i max(q_i hi_i, q_i lo_i) for every key between a page's
// bounds, channel by channel.  Bounds are 8-bit whole numbers times a power of
// two, rounded outwards, and queries 8-bit whole numbers times a power of two, so
// a score is a whole number below 2^21 times a power of two: exact in fp32, in
// whatever order it is summed, and the pages chosen do not depend on the kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

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
// Bounds.  One CTA per (page, KV head); a page is at most 32 KB and is read in
// one go, so that all of its loads are in flight at once.
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

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int V = FP8 ? 16 : 8;     // values of a 16-byte vector
    constexpr int LPR = D / V;          // lanes per row
    constexpr int RW = 32 / LPR;        // rows per load of a warp
    constexpr int STEP = RW * kBoundsWarps;
    constexpr int U = 8;
    __shared__ float part[kBoundsWarps][2][D];
    __shared__ float red[kBoundsWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = blockIdx.y, b = blockIdx.z;
    bool bad;
    const int L = clamp_seq_len(a.lens[b], a.P, a.max_pages, bad);
    const int start = a.starts != nullptr ? a.starts[b] : 0;
    if (bad || start < 0) {
        if (tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
        return;
    }
    const int end = start < L ? (L + a.P - 1) / a.P : 0;
    const int sub = lane % LPR, row0 = warp * RW + lane / LPR;
    for (int j = start / a.P + blockIdx.x; j < end; j += gridDim.x) {
        const int page = a.table[static_cast<size_t>(b) * a.max_pages + j];
        if (page < 0 || page >= a.num_pages) {
            if (tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            continue;
        }
        const int n = min(a.P, L - j * a.P);
        const size_t first = (static_cast<size_t>(page) * a.Hkv + hk) * a.P;  // row of the pool
        float hi[V], lo[V];
        if (FP8) {
            const uint8_t* base = static_cast<const uint8_t*>(a.k_pages) + first * D + sub * 16;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                hi[i] = -INFINITY;
                lo[i] = INFINITY;
            }
            for (int r0 = row0; r0 < n + row0; r0 += U * STEP) {
                uint4 x[U];
                uint8_t s[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * STEP;
                    if (r < n) {
                        x[u] = ptx::ld_stream(base + static_cast<size_t>(r) * D);
                        s[u] = a.k_scales[first + r];
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (r0 + u * STEP >= n) break;
                    const float f = scale_of(s[u]);
                    const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[2];
                        f16x2_of_e4m3x4(w[i], h[0], h[1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 y = __half22float2(*reinterpret_cast<__half2*>(&h[k]));
                            const int at = i * 4 + k * 2;
                            hi[at] = fmaxf(hi[at], y.x * f);
                            lo[at] = fminf(lo[at], y.x * f);
                            hi[at + 1] = fmaxf(hi[at + 1], y.y * f);
                            lo[at + 1] = fminf(lo[at + 1], y.y * f);
                        }
                    }
                }
            }
        } else {
            const uint16_t* base = static_cast<const uint16_t*>(a.k_pages) + first * D + sub * 8;
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
                    for (int i = 0; i < 4; ++i) {  // (the number, of a number and a NaN)
                        h[i] = max_bf16x2(h[i], w[i]);
                        l[i] = min_bf16x2(l[i], w[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[2 * i] = __uint_as_float(h[i] << 16);
                hi[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
                lo[2 * i] = __uint_as_float(l[i] << 16);
                lo[2 * i + 1] = __uint_as_float(l[i] & 0xffff0000u);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int off = LPR; off < 32; off <<= 1) {
                hi[i] = fmaxf(hi[i], __shfl_xor_sync(kFull, hi[i], off));
                lo[i] = fminf(lo[i], __shfl_xor_sync(kFull, lo[i], off));
            }
        }
        __syncthreads();  // (the page before has been read from `part`)
        if (lane < LPR) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[warp][0][sub * V + i] = hi[i];
                part[warp][1][sub * V + i] = lo[i];
            }
        }
        __syncthreads();
        float h = 0.0f, l = 0.0f;
        if (tid < D) {
            h = part[0][0][tid];
            l = part[0][1][tid];
#pragma unroll
            for (int w = 1; w < kBoundsWarps; ++w) {
                h = fmaxf(h, part[w][0][tid]);
                l = fminf(l, part[w][1][tid]);
            }
            if (!(h >= l)) h = l = 0.0f;  // no number at all
            const float most = __uint_as_float(0x7f7f0000u);
            h = fminf(fmaxf(h, -most), most);
            l = fminf(fmaxf(l, -most), most);
        }
        float top = fmaxf(fabsf(h), fabsf(l));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        top = red[0];
#pragma unroll
        for (int w = 1; w < kBoundsWarps; ++w) top = fmaxf(top, red[w]);
        const int e = exponent_for(top);
        const float inv = pow2(-e);
        const size_t at = static_cast<size_t>(page) * a.Hkv + hk;
        if (tid < D) {
            a.bounds[at * 2 * D + tid] =
                static_cast<int8_t>(fminf(fmaxf(ceilf(h * inv), -127.0f), 127.0f));
            a.bounds[at * 2 * D + D + tid] =
                static_cast<int8_t>(fminf(fmaxf(floorf(l * inv), -127.0f), 127.0f));
        }
        if (tid == 0) a.exps[at] = static_cast<uint8_t>(e + 127);
    }
}

// ---------------------------------------------------------------------------
// Selection.  A cluster of CTAs takes the pages of one (sequence, KV head) for
// some of its tokens.  With p = max(c, 0) and m = min(c, 0) a score is
// p . hi + m . lo: a product of the pages' bounds (16 pages to a tile, 2 d deep)
// with the query codes, on the tensor cores in fp16, whose products and fp32 sums
// of such whole numbers are exact.  The highest scores are then found by their
// bits, eight at a time from the top, and written in the order of the pages.
//
// The bounds of a page are contiguous and each is used once, so they go from
// memory straight into the product's registers: the order of channels within a
// product is free, and is chosen so that a lane's 16 bytes are its operand.
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
    int32_t* status;
};

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kTilesAtOnce = 4;  // column tiles that share one conversion of the bounds

// Order-preserving bits of a score; 0 for a page that scores nothing.
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

__device__ __forceinline__ uint32_t max0_f16x2(uint32_t x) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0u));
    return r;
}
__device__ __forceinline__ uint32_t min0_f16x2(uint32_t x) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0u));
    return r;
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

// By NW warps (all of the CTA, or each warp for itself): the k highest of n keys,
// as ascending indices to out[0 .. k).
template <int NW>
__device__ __forceinline__ void take_highest(const Keys& key, int n, int k, int32_t* out,
                                             int* hist, int* counts, int t) {
    constexpr int GS = 32 * NW;
    auto sync = [] {
        if (NW > 1)
            __syncthreads();
        else
            __syncwarp();
    };
    const int lane = t & 31, w = t >> 5;
    uint32_t prefix = 0, known = 0;
    int left = k;  // still to be found among the keys that share the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = t; i < 256; i += GS) hist[i] = 0;
        sync();
        for (int i = t; i < n; i += GS) {
            const uint32_t v = key(i);
            if ((v & known) == prefix) atomicAdd(hist + ((v >> shift) & 255u), 1);
        }
        sync();
        // The bin that holds the left-th from the top; every warp finds it.
        int own = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) own += hist[255 - (lane * 8 + j)];
        int upto = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(kFull, upto, off);
            if (lane >= off) upto += y;
        }
        const int src = __ffs(__ballot_sync(kFull, upto >= left)) - 1;
        int above = upto - own, bin = 0;
        if (lane == src) {
            int j = 0;
            for (; j < 7; ++j) {
                const int c = hist[255 - (lane * 8 + j)];
                if (above + c >= left) break;
                above += c;
            }
            bin = 255 - (lane * 8 + j);
        }
        bin = __shfl_sync(kFull, bin, src);
        left -= __shfl_sync(kFull, above, src);
        prefix |= static_cast<uint32_t>(bin) << shift;
        known |= 255u << shift;
        sync();  // (hist is read)
    }
    // Keys above the prefix, and the first `left` that equal it.
    const int seg = ((n + GS - 1) / GS) * 32;  // of one warp
    const int lo = min(w * seg, n), hi = min(lo + seg, n);
    int more = 0, same = 0;
    if (NW > 1) {
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const uint32_t v = i0 + lane < hi ? key(i0 + lane) : 0u;
            more += __popc(__ballot_sync(kFull, i0 + lane < hi && v > prefix));
            same += __popc(__ballot_sync(kFull, i0 + lane < hi && v == prefix));
        }
        if (lane == 0) {
            counts[2 * w] = more;
            counts[2 * w + 1] = same;
        }
        sync();
        more = same = 0;
        for (int i = 0; i < w; ++i) {
            more += counts[2 * i];
            same += counts[2 * i + 1];
        }
    }
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const uint32_t v = i0 + lane < hi ? key(i0 + lane) : 0u;
        const unsigned gt = __ballot_sync(kFull, i0 + lane < hi && v > prefix);
        const unsigned eq = __ballot_sync(kFull, i0 + lane < hi && v == prefix);
        const unsigned below = (1u << lane) - 1u;
        const int eq_rank = same + __popc(eq & below);
        const bool take = ((gt >> lane) & 1u) != 0 || (((eq >> lane) & 1u) != 0 && eq_rank < left);
        if (take) out[more + __popc(gt & below) + min(eq_rank, left)] = i0 + lane;
        more += __popc(gt);
        same += __popc(eq);
    }
    sync();
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kStride = D + 4;  // halves: lanes g of a fragment load fall on banks of their own
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int S = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    const int unit = blockIdx.x / S;
    const int hk = unit / a.chunks % a.Hkv, b = unit / (a.chunks * a.Hkv);
    const int t0 = unit % a.chunks * a.TC;
    const int nt = min(a.TC, a.T - t0);  // tokens
    const int G = a.Hq / a.Hkv;
    const int tiles = (a.TC * a.cols + 7) / 8;
    uint32_t* scores = reinterpret_cast<uint32_t*>(smem);  // [TC][per_most]
    int* hist = reinterpret_cast<int*>(scores + static_cast<size_t>(a.TC) * a.per_most);
    int* counts = hist + 256 * kSelWarps;
    __half* codes = reinterpret_cast<__half*>(counts + 2 * kSelWarps);  // [tiles * 8][kStride]

    bool bad;
    const int L = clamp_seq_len(a.lens[b], a.P, a.max_pages, bad);
    if (bad && tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    const int nb = (L + a.P - 1) / a.P;
    const int per = max((nb + S - 1) / S, 1);
    const int lo = min(rank * per, nb), hi = min(lo + per, nb);

    if (nb > a.n_select) {
        // Query codes: a warp takes a token's heads.
        for (int t = warp; t < tiles * 8 / a.cols; t += kSelWarps) {
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
            for (int i = lane; i < a.cols * D; i += 32) {
                const int col = i / D, d = i % D;  // columns past the group repeat its first head
                const float x = __uint_as_float(
                    static_cast<uint32_t>(q[(col < G ? col : 0) * D + d]) << 16);
                const float y = x != x ? 0.0f : fminf(fmaxf(rintf(x * inv), -127.0f), 127.0f);
                codes[static_cast<size_t>(t * a.cols + col) * kStride + d] = __float2half_rn(y);
            }
        }
        __syncthreads();
        constexpr int NC = D / 64;  // 16-byte vectors of a row of bounds, to a lane
        const int32_t* table = a.table + static_cast<size_t>(b) * a.max_pages;
        for (int p0 = lo + warp * 16; p0 < hi; p0 += kSelWarps * 16) {
            uint4 x[2][2][NC];  // [page g, g + 8][hi, lo]
            float size[2];
            bool none[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                int page = table[min(p0 + g + 8 * r, hi - 1)];
                none[r] = page < 0 || page >= a.num_pages;
                if (none[r]) {
                    report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                    page = 0;
                }
                const size_t at = static_cast<size_t>(page) * a.Hkv + hk;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < NC; ++j)
                        x[r][h][j] = ptx::ld_stream(a.bounds + at * 2 * D + h * D + j * 64 + c * 16);
                size[r] = scale_of(a.exps[at]);
            }
            __syncwarp();
            for (int n0 = 0; n0 < tiles; n0 += kTilesAtOnce) {
                float acc[kTilesAtOnce][4];
#pragma unroll
                for (int n = 0; n < kTilesAtOnce; ++n)
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
                        for (int n = 0; n < kTilesAtOnce; ++n) {
                            if (n0 + n >= tiles) break;
                            const uint2 q = *reinterpret_cast<const uint2*>(
                                codes + static_cast<size_t>((n0 + n) * 8 + g) * kStride + j * 64 +
                                c * 16 + w * 4);
                            ptx::mma_sync_f16(acc[n], f[0][0], f[0][1], f[0][2], f[0][3],
                                              max0_f16x2(q.x), max0_f16x2(q.y));
                            ptx::mma_sync_f16(acc[n], f[1][0], f[1][1], f[1][2], f[1][3],
                                              min0_f16x2(q.x), min0_f16x2(q.y));
                        }
                    }
                }
                // The largest of each token's columns.
#pragma unroll
                for (int n = 0; n < kTilesAtOnce; ++n) {
                    if (n0 + n >= tiles) break;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float y0 = acc[n][2 * r], y1 = acc[n][2 * r + 1];
                        if (a.cols > 1) y0 = fmaxf(y0, y1);
                        if (a.cols > 2) y0 = fmaxf(y0, __shfl_xor_sync(kFull, y0, 1));
                        if (a.cols > 4) y0 = fmaxf(y0, __shfl_xor_sync(kFull, y0, 2));
                        const int i = p0 + g + 8 * r;
                        const bool forced = i < a.n_first || i >= nb - a.n_last;
                        auto put = [&](int t, float y, bool again) {
                            if (i >= hi || t >= nt) return;
                            uint32_t* to = scores + static_cast<size_t>(t) * a.per_most + (i - lo);
                            const uint32_t k =
                                forced ? 0xffffffffu : none[r] ? 0u : score_key(y * size[r]);
                            *to = again ? max(*to, k) : k;
                        };
                        const int col = (n0 + n) * 8 + 2 * c;
                        if (a.cols == 1) {
                            put(col, y0, false);
                            put(col + 1, y1, false);
                        } else if (2 * c % (a.cols < 8 ? a.cols : 8) == 0) {
                            put(col / a.cols, y0, col % a.cols != 0);
                        }
                    }
                }
            }
        }
    }
    if (S > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    // Tokens are shared out over the cluster's CTAs, and within a CTA over its
    // warps where there are several.
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
    if (nb > a.n_select) {
        if (nt > S) {
            for (int t = rank + S * warp; t < nt; t += S * kSelWarps) {
                key.at = ptx::smem_u32(scores + static_cast<size_t>(t) * a.per_most);
                take_highest<1>(key, nb, k, row_of(t), hist + 256 * warp, counts, lane);
            }
        } else if (rank < nt) {
            key.at = ptx::smem_u32(scores + static_cast<size_t>(rank) * a.per_most);
            take_highest<kSelWarps>(key, nb, k, row_of(rank), hist, counts, tid);
        }
    }
    if (S > 1) ptx::cluster_sync();  // (other CTAs may still read this one's scores)
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

bool cache_shape_ok(int B, int Hkv, int d, int max_pages, int P, int num_pages) {
    return B >= 0 && B <= 65535 && Hkv >= 1 && Hkv <= 65535 && (d == 64 || d == 128) &&
           max_pages >= 1 && num_pages >= 1 && page_size_ok(P) &&
           static_cast<long long>(num_pages) * Hkv * P < (1LL << 31) &&
           static_cast<long long>(max_pages) * P < (1LL << 31);
}

constexpr int kMaxSelectPages = 262144;

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_kv_block_bounds(const void* k_pages, const uint8_t* k_scales, const int32_t* block_table,
                         int max_pages_per_seq, const int32_t* starts, const int32_t* seq_lens,
                         int8_t* bounds, uint8_t* bounds_exp, int B, int Hkv, int d,
                         int page_size, int num_pages, int32_t* status, void* stream) {
    if (!cache_shape_ok(B, Hkv, d, max_pages_per_seq, page_size, num_pages))
        return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    if (!k_pages || !block_table || !seq_lens || !bounds || !bounds_exp) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(k_pages, 16) || !ptr_aligned(bounds, 16) || !ptr_aligned(block_table, 4) ||
        !ptr_aligned(starts, 4) || !ptr_aligned(seq_lens, 4) || !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    const int sms = sm_count();
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
    // The host does not know how many pages a sequence has: its CTAs take them in
    // turn, twelve to an SM where there are that many.
    const long long rows = static_cast<long long>(B) * Hkv;
    const long long fill = (12LL * sms + rows - 1) / rows;
    const int nx = static_cast<int>(fill < max_pages_per_seq ? fill : max_pages_per_seq);
    using Kernel = void (*)(BoundsArgs);
    const Kernel kernel = k_scales ? (d == 128 ? bounds_kernel<128, true> : bounds_kernel<64, true>)
                                   : (d == 128 ? bounds_kernel<128, false>
                                               : bounds_kernel<64, false>);
    return rc_of(launch_dependent(kernel, dim3(nx, Hkv, B), dim3(kBoundsThreads), 0,
                                  static_cast<cudaStream_t>(stream), a));
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
    const int sms = sm_count();
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
    const size_t code_row = static_cast<size_t>(d + 4) * 2;
    int TC = T;
    size_t need = 0;
    for (;; TC = (TC + 1) / 2) {
        a.per_most = ((max_pages_per_seq + S - 1) / S + 3) / 4 * 4;
        need = static_cast<size_t>(TC) * a.per_most * 4 + (256 + 2) * kSelWarps * 4 +
               static_cast<size_t>((TC * a.cols + 7) / 8 * 8) * code_row;
        if (need <= (TC == 1 ? 200u * 1024u : 100u * 1024u)) break;
        if (TC == 1) {  // one token of a very long sequence: more CTAs share its pages
            if (S == 8) return TREE_ATTN_ERR_SHAPE;
            S *= 2;
            TC = 2;  // (1 again)
        }
    }
    a.TC = TC;
    a.chunks = (T + TC - 1) / TC;
    const long long grid = static_cast<long long>(B) * Hkv * a.chunks * S;
    if (grid >= (1LL << 31)) return TREE_ATTN_ERR_SHAPE;
    using Kernel = void (*)(SelectArgs);
    const Kernel kernel = d == 128 ? select_kernel<128> : select_kernel<64>;
    if (need > 48 * 1024 &&
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(need)) != cudaSuccess)
        return TREE_ATTN_ERR_CUDA;
    return rc_of(launch_cluster(kernel, dim3(static_cast<unsigned>(grid)), dim3(kSelThreads), need,
                                S, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
