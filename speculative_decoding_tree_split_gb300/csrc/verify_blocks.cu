// verify_blocks.cu -- split tree attention over selected pages of a bf16 or 8-bit
// cache (one token per sequence: sparse decoding).
//
// Every (sequence, token, KV head) has its own list of pages, so the query rows
// that share keys are the G heads of a group: at most 8 or 16 rows, and the work
// is reading the pages.  A unit (those rows and their list) is split over the
// CTAs of a cluster and the warps of a CTA, 16 keys to a tile; each warp keeps
// running maxima, sums and accumulators of its own, which the CTA joins through
// shared memory and the cluster through one another's, so there is one launch and
// no workspace.
//
// K and V go from memory straight into the registers of the product: with
// S^T = K Q^T and O^T = V^T P^T the keys (channels) are the 16-row side and the
// query rows the 8-column side, so no half of a tile is padding for G <= 8, and
// since the order of channels within the product is free, it is chosen so that 16
// contiguous bytes of a row are a lane's operands.  V's pairs of keys are put
// together by byte permutes, P turns from result to operand by movmatrix.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
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
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;        // keys
constexpr float kMove = 8.0f;    // binades a score may exceed its row's reference by
// 8-bit cache: P's largest at a fresh reference is 2^kLift (2^8 above it is still
// below fp16's 2^16).
constexpr int kLift = 6;
constexpr int kNoScale = -1000;  // no key has been seen

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

struct Args {
    const uint16_t* q;
    const void* kv[2];        // K, V pools
    const uint8_t* scales[2];
    const int32_t* table;
    const int32_t* lens;
    const int32_t* blocks;
    const uint16_t* tree[2];
    const uint64_t* mask;
    const int32_t* parents;
    uint16_t* out;
    float* lse;
    int n_blocks, max_pages, mask_stride, parents_stride, Hq, Hkv, T, P, num_pages, row_blocks;
    float scale_log2;
    int32_t* status;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^e for any e that fp32 holds, 0 below.
__device__ __forceinline__ float pow2(int e) {
    return e < -126 ? 0.0f : __int_as_float((min(e, 127) + 127) << 23);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One warp's running state for NT * 8 query rows; a lane holds columns 2c and
// 2c + 1 of every column tile.
template <int D, int NT>
struct State {
    float m[NT][2];           // references, in units of log2
    float l[NT][2];           // this lane's part of the sums
    float o[NT][D / 16][4];   // [column tile][channel tile]
};

// Moves the references where a score exceeds one by more than kMove.
template <int D, int NT>
__device__ __forceinline__ void follow(State<D, NT>& st, const float (&x)[NT][4]) {
    bool move = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) move |= x[n][i] > st.m[n][i & 1] + kMove;
    if (!__any_sync(kFull, move)) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float t = fmaxf(x[n][i], x[n][i + 2]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
                t = fmaxf(t, __shfl_xor_sync(kFull, t, off));
            t = fmaxf(t, st.m[n][i]);
            f[i] = st.m[n][i] == -INFINITY ? 0.0f : ex2(st.m[n][i] - t);
            st.m[n][i] = t;
            st.l[n][i] *= f[i];
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][d][i] *= f[i & 1];
    }
}

// Scores to probabilities (in place), summed.
template <int D, int NT>
__device__ __forceinline__ void exponents(State<D, NT>& st, float (&x)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float m = st.m[n][i & 1];
            x[n][i] = ex2(x[n][i] - (m == -INFINITY ? 0.0f : m));
            st.l[n][i & 1] += x[n][i];
        }
}

// O^T += V^T P^T for 16 keys of bf16 values, the probabilities (times f) as two
// bf16 numbers: what one leaves out (2^-9) would be the largest error before the
// result is rounded, and the product is not what bounds the kernel.
template <int D, int NT>
__device__ __forceinline__ void add_values_bf16(State<D, NT>& st, const float (&p)[NT][4],
                                                const uint4 (&v)[4][D / 64], float f) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float y[4];
        uint32_t b[2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = p[n][i] * f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t hi = pack_bf16(y[2 * h], y[2 * h + 1]);
            const uint32_t lo = pack_bf16(y[2 * h] - __uint_as_float(hi << 16),
                                          y[2 * h + 1] - __uint_as_float(hi & 0xffff0000u));
            b[0][h] = ptx::transpose8(hi);
            b[1][h] = ptx::transpose8(lo);
        }
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t k0 = word(v[0][h], w), k1 = word(v[1][h], w);
                const uint32_t k2 = word(v[2][h], w), k3 = word(v[3][h], w);
                const uint32_t a0 = __byte_perm(k0, k1, 0x5410), a1 = __byte_perm(k0, k1, 0x7632);
                const uint32_t a2 = __byte_perm(k2, k3, 0x5410), a3 = __byte_perm(k2, k3, 0x7632);
                ptx::mma_sync_bf16(st.o[n][h * 4 + w], a0, a1, a2, a3, b[0][0], b[0][1]);
                ptx::mma_sync_bf16(st.o[n][h * 4 + w], a0, a1, a2, a3, b[1][0], b[1][1]);
            }
    }
}

// Channel of o[.][t][0 or 1] (the next one for 2 and 3) of lane g.
template <int D>
__device__ __forceinline__ int channel_bf16(int t, int g) {
    return (t / 4) * 64 + 8 * g + 2 * (t % 4);
}
template <int D>
__device__ __forceinline__ int channel_fp8(int t, int g) {
    return (D / 8) * g + 2 * t;
}

// 16 bf16 keys: the lane's vectors of rows g and g + 8, and of the values of rows
// 2c, 2c + 1, 2c + 8, 2c + 9, by a function from row to address.
template <int D, typename Row>
__device__ __forceinline__ void load_keys_bf16(uint4 (&k)[2][D / 32], Row row, int g, int c) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) k[r][j] = ptx::ld_stream(row(g + 8 * r) + j * 32 + c * 8);
}
template <int D, typename Row>
__device__ __forceinline__ void load_values_bf16(uint4 (&v)[4][D / 64], Row row, int g, int c) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            v[r][h] = ptx::ld_stream(row(2 * c + (r & 1) + 8 * (r >> 1)) + h * 64 + g * 8);
}

template <int D, int NT>
__device__ __forceinline__ void scores_bf16(float (&x)[NT][4], const uint4 (&k)[2][D / 32],
                                            const uint4 (&q)[NT][D / 32]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            ptx::mma_sync_bf16(x[n], k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y, q[n][j].x,
                               q[n][j].y);
            ptx::mma_sync_bf16(x[n], k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w, q[n][j].z,
                               q[n][j].w);
        }
    }
}

template <int NT>
__device__ __forceinline__ void hide(float (&x)[NT][4], int live, int g) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (g >= live) x[n][0] = x[n][1] = -INFINITY;
        if (g + 8 >= live) x[n][2] = x[n][3] = -INFINITY;
    }
}

// A probability of 0 times a value that is no number is no number, so values of
// keys that are not there are cleared.
template <int N>
__device__ __forceinline__ void clear_values(uint4 (&v)[4][N], int live, int c) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (2 * c + (r & 1) + 8 * (r >> 1) >= live)
#pragma unroll
            for (int h = 0; h < N; ++h) v[r][h] = make_uint4(0u, 0u, 0u, 0u);
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) blocks_kernel(const Args a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int R = 8 * NT;        // query rows
    constexpr int kStride = D + 4;   // floats of a partial row
    float* part = reinterpret_cast<float*>(smem);             // [kWarps][R][kStride]
    float* part_m = part + kWarps * R * kStride;              // [kWarps][R]
    float* part_l = part_m + kWarps * R;                      // [kWarps][R]
    float* mine = part_l + kWarps * R;                        // [R][kStride] the CTA's own
    float* mine_m = mine + R * kStride;                       // [R], then l [R]
    int* pages = reinterpret_cast<int*>(mine_m + 2 * R);      // [n_blocks] rows of the pool, or -1
    int* live_of = pages + a.n_blocks;                        // [n_blocks] committed tokens
    __shared__ int8_t seen[TREE_ATTN_MAX_T];                  // tree tokens that the mask allows
    __shared__ int n_seen, n_used;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int S = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    // Units in the order (sequence, KV head, token): tokens share most pages.
    int unit = blockIdx.x / S;
    const int rb = unit % a.row_blocks;
    unit /= a.row_blocks;
    const int t = unit % a.T;
    unit /= a.T;
    const int hk = unit % a.Hkv, b = unit / a.Hkv;
    const int G = a.Hq / a.Hkv;
    const int rows = min(G - rb * R, R);
    const size_t token = static_cast<size_t>(b) * a.T + t;
    const size_t row0 = token * a.Hq + static_cast<size_t>(hk) * G + rb * R;  // of q and out

    // The page list, and the tree tokens that t sees.
    bool bad;
    const int L = clamp_seq_len(a.lens[b], a.P, a.max_pages, bad);
    if (bad && tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    const int nb = (L + a.P - 1) / a.P;
    if (tid == 0) n_used = 0;
    __syncthreads();
    const int32_t* list = a.blocks + (token * a.Hkv + hk) * a.n_blocks;
    for (int i = tid; i < a.n_blocks; i += kThreads) {
        const int j = list[i];
        int page = -1;
        if (j >= 0 && j < nb) page = a.table[static_cast<size_t>(b) * a.max_pages + j];
        if (page < 0 || page >= a.num_pages) {
            if (j != -1) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            page = -1;
        }
        pages[i] = page;
        live_of[i] = page < 0 ? 0 : min(a.P, L - j * a.P);
        if (page >= 0) atomicMax(&n_used, i + 1);
    }
    if (warp == 0) {
        uint64_t bits = 0;
        if (a.mask != nullptr) {
            bits = a.mask[static_cast<size_t>(b) * a.mask_stride + t];
            if (a.T < 64) bits &= (1ull << a.T) - 1ull;
        } else {
            const int32_t* up = a.parents + static_cast<size_t>(b) * a.parents_stride;
            const int p0 = lane < a.T ? up[lane] : -1, p1 = lane + 32 < a.T ? up[lane + 32] : -1;
            if (p0 < -1 || (p0 >= lane && lane < a.T) || p1 < -1 ||
                (p1 >= lane + 32 && lane + 32 < a.T))
                report(a.status, TREE_ATTN_STATUS_BAD_PARENT);
            int j = t;
            while (j >= 0) {
                bits |= 1ull << j;
                const int q0 = __shfl_sync(kFull, p0, j & 31), q1 = __shfl_sync(kFull, p1, j & 31);
                const int p = j < 32 ? q0 : q1;
                j = p < j ? p : -1;  // (towards the root, whatever the array holds)
            }
        }
        for (int h = 0; h < 2; ++h) {
            const int j = lane + 32 * h;
            if ((bits >> j) & 1ull)
                seen[__popcll(bits & ((1ull << j) - 1ull))] = static_cast<int8_t>(j);
        }
        if (lane == 0) n_seen = __popcll(bits);
    }

    // Queries as the product's second operand: row g of each column tile.
    uint4 q[NT][D / 32];
    float rf[NT][2];  // per column: score unit (8-bit cache: with the row's power of two)
    auto load_q = [&] {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + g;
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                q[n][j] = r < rows ? *reinterpret_cast<const uint4*>(
                                         a.q + (row0 + r) * D + j * 32 + c * 8)
                                   : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    if (FP8) {
        // fp16, scaled so that the row's largest lies in [2^14, 2^15): exact down to
        // 2^-28 of it, and to 2^-39 of it below.  The order of channels is that of the
        // 8-bit rows: 16 to a lane.
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + g;
            const uint16_t* from = a.q + (row0 + (r < rows ? r : 0)) * D;
            uint4 raw[D / 64][2];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    raw[j][h] =
                        *reinterpret_cast<const uint4*>(from + j * 64 + c * 16 + h * 8);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t x = word(raw[j][h], w);
                        const uint32_t lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
                        top = max(top, lo < 0x7f80u ? lo : 0u);
                        top = max(top, hi < 0x7f80u ? hi : 0u);
                    }
                }
            top = max(top, __shfl_xor_sync(kFull, top, 1));
            top = max(top, __shfl_xor_sync(kFull, top, 2));
            const int e = max(static_cast<int>(top >> 7) - 127 - 14, -112);  // exponent of the unit
            const float inv = pow2(-e);
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t y[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t x = word(raw[j][h], w);
                        y[w] = pack_f16(__uint_as_float(x << 16) * inv,
                                        __uint_as_float(x & 0xffff0000u) * inv);
                    }
                    q[n][j * 2 + h] = r < rows ? make_uint4(y[0], y[1], y[2], y[3])
                                               : make_uint4(0u, 0u, 0u, 0u);
                }
            // Lanes hold row g's exponent, and need those of rows 2c and 2c + 1.
#pragma unroll
            for (int i = 0; i < 2; ++i)
                rf[n][i] = pow2(__shfl_sync(kFull, e, (2 * c + i) * 4)) * a.scale_log2;
        }
    } else {
        load_q();
#pragma unroll
        for (int n = 0; n < NT; ++n) rf[n][0] = rf[n][1] = a.scale_log2;
    }

    State<D, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            st.m[n][i] = -INFINITY;
            st.l[n][i] = 0.0f;
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][d][i] = 0.0f;
    }
    int sref = kNoScale;  // 8-bit cache: accumulators are in units of 2^(sref - kLift)
    __syncthreads();

    const int per_page = a.P / kTile, shift = __ffs(per_page) - 1;
    const int tiles = n_used << shift;
    const int step = S * kWarps;
    const int w0 = rank * kWarps + warp;
    if (!FP8) {
        uint4 k[2][D / 32], v[4][D / 64];
        // The tile's first row in the pools, and its keys.
        auto find = [&](int i, size_t& first) {
            const int e = i >> shift, off = (i & (per_page - 1)) * kTile;
            first = (static_cast<size_t>(max(pages[e], 0)) * a.Hkv + hk) * a.P + off;
            return min(max(live_of[e] - off, 0), kTile);
        };
        auto load_k = [&](size_t first) {
            const uint16_t* base = static_cast<const uint16_t*>(a.kv[0]) + first * D;
            load_keys_bf16<D>(k, [&](int r) { return base + r * D; }, g, c);
        };
        auto load_v = [&](size_t first) {
            const uint16_t* base = static_cast<const uint16_t*>(a.kv[1]) + first * D;
            load_values_bf16<D>(v, [&](int r) { return base + r * D; }, g, c);
        };
        int i = w0, live = 0;
        size_t first = 0;
        // (tiles without keys are passed over)
        auto next = [&](int from) {
            live = 0;
            for (i = from; i < tiles; i += step)
                if ((live = find(i, first)) > 0) break;
        };
        next(w0);
        if (live > 0) {
            load_k(first);
            load_v(first);
        }
        while (live > 0) {
            float x[NT][4];
            scores_bf16<D, NT>(x, k, q);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] *= rf[n][j & 1];
            const int now = live;
            next(i + step);
            if (live > 0) load_k(first);
            if (now < kTile) {
                hide<NT>(x, now, g);
                clear_values(v, now, c);
            }
            follow(st, x);
            exponents(st, x);
            add_values_bf16<D, NT>(st, x, v, 1.0f);
            if (live > 0) load_v(first);
        }
    } else {
        constexpr int NC = D / 64;
        uint4 k[2][NC];
        uint4 v[4];
        uint32_t s[2][2];  // [K, V] scale bytes of keys g and g + 8
        auto find = [&](int i, size_t& first) {
            const int e = i >> shift, off = (i & (per_page - 1)) * kTile;
            first = (static_cast<size_t>(max(pages[e], 0)) * a.Hkv + hk) * a.P + off;
            return min(max(live_of[e] - off, 0), kTile);
        };
        auto load_k = [&](size_t first) {
            const uint8_t* base = static_cast<const uint8_t*>(a.kv[0]) + first * D + c * 16;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int j = 0; j < NC; ++j) k[r][j] = ptx::ld_stream(base + (g + 8 * r) * D + j * 64);
                s[0][r] = a.scales[0][first + g + 8 * r];
            }
        };
        auto load_v = [&](size_t first) {
            const uint8_t* base = static_cast<const uint8_t*>(a.kv[1]) + first * D + g * (D / 8);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint8_t* p = base + (2 * c + (r & 1) + 8 * (r >> 1)) * D;
                if (D == 128) {
                    v[r] = ptx::ld_stream(p);
                } else {
                    const uint2 y = ptx::ld_stream8(p);
                    v[r] = make_uint4(y.x, y.y, 0u, 0u);
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) s[1][r] = a.scales[1][first + g + 8 * r];
        };
        int i = w0, live = 0;
        size_t first = 0;
        auto next = [&](int from) {
            live = 0;
            for (i = from; i < tiles; i += step)
                if ((live = find(i, first)) > 0) break;
        };
        next(w0);
        if (live > 0) {
            load_k(first);
            load_v(first);
        }
        while (live > 0) {
            float x[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t f[4];
                    f16x2_of_e4m3x4(word(k[0][j], w), f[0], f[2]);
                    f16x2_of_e4m3x4(word(k[1][j], w), f[1], f[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 y = q[n][2 * j + w / 2];
                        ptx::mma_sync_f16(x[n], f[0], f[1], f[2], f[3], w % 2 ? y.z : y.x,
                                          w % 2 ? y.w : y.y);
                    }
                }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] = x[n][j] * scale_of(s[0][j >> 1]) * rf[n][j & 1];
            const int now = live;
            next(i + step);
            if (live > 0) load_k(first);
            int sv[2] = {static_cast<int>(s[1][0]) - 127, static_cast<int>(s[1][1]) - 127};
            if (now < kTile) {
                hide<NT>(x, now, g);
                if (g >= now) sv[0] = kNoScale;
                if (g + 8 >= now) sv[1] = kNoScale;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (2 * c + (r & 1) + 8 * (r >> 1) >= now) v[r] = make_uint4(0u, 0u, 0u, 0u);
            }
            follow(st, x);
            exponents(st, x);
            // The unit of the accumulators follows the largest value scale.
            const int top = __reduce_max_sync(kFull, max(sv[0], sv[1]));
            if (top > sref) {
                const float f = sref == kNoScale ? 1.0f : pow2(sref - top);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
#pragma unroll
                        for (int j = 0; j < 4; ++j) st.o[n][d][j] *= f;
                sref = top;
            }
            const float pf[2] = {pow2(sv[0] - sref + kLift), pow2(sv[1] - sref + kLift)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t b0 = ptx::transpose8(pack_f16(x[n][0] * pf[0], x[n][1] * pf[0]));
                const uint32_t b1 = ptx::transpose8(pack_f16(x[n][2] * pf[1], x[n][3] * pf[1]));
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    const uint32_t k0 = word(v[0], w), k1 = word(v[1], w);
                    const uint32_t k2 = word(v[2], w), k3 = word(v[3], w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // channels 4w + 2h and the next
                        uint32_t a0, a1, a2, a3;
                        f16x2_of_e4m3x4(__byte_perm(k0, k1, h ? 0x7362 : 0x5140), a0, a1);
                        f16x2_of_e4m3x4(__byte_perm(k2, k3, h ? 0x7362 : 0x5140), a2, a3);
                        ptx::mma_sync_f16(st.o[n][2 * w + h], a0, a1, a2, a3, b0, b1);
                    }
                }
            }
            if (live > 0) load_v(first);
        }
    }
    // Tree tokens: tiles behind the pages' (bf16 in either cache).
    {
        const int n = n_seen;
        const size_t stride = static_cast<size_t>(a.Hkv) * D;
        const size_t base = (static_cast<size_t>(b) * a.T * a.Hkv + hk) * D;
        for (int i = 0; i * kTile < n; ++i) {
            if ((tiles + i) % step != w0) continue;
            const int live = min(n - i * kTile, kTile);
            auto at = [&](const uint16_t* p, int r) {
                return p + base + seen[i * kTile + min(r, live - 1)] * stride;
            };
            uint4 k[2][D / 32], v[4][D / 64];
            load_keys_bf16<D>(k, [&](int r) { return at(a.tree[0], r); }, g, c);
            if (FP8) load_q();
            float x[NT][4];
            scores_bf16<D, NT>(x, k, q);
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[m][j] *= a.scale_log2;
            hide<NT>(x, live, g);
            follow(st, x);
            exponents(st, x);
            if (FP8 && sref == kNoScale) sref = 0;
            // The value operand's channels follow the accumulators' order.
            if (FP8) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint16_t* p = at(a.tree[1], 2 * c + (r & 1) + 8 * (r >> 1)) + g * (D / 8);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) v[r][h] = ptx::ld_stream(p + 8 * h);
                }
            } else {
                load_values_bf16<D>(v, [&](int r) { return at(a.tree[1], r); }, g, c);
            }
            clear_values(v, live, c);
            add_values_bf16<D, NT>(st, x, v, FP8 ? pow2(kLift - sref) : 1.0f);
        }
    }

    // This warp's rows to shared memory.
    const float unit_of = FP8 && sref != kNoScale ? pow2(sref - kLift) : 1.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float l = st.l[n][i];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);
            const int r = n * 8 + 2 * c + i;
            if (g == 0) {
                part_m[warp * R + r] = st.m[n][i];
                part_l[warp * R + r] = l;
            }
            float* to = part + (warp * R + r) * kStride;
#pragma unroll
            for (int d = 0; d < D / 16; d += 2) {
                const int ch = FP8 ? channel_fp8<D>(d, g) : channel_bf16<D>(d, g);
                *reinterpret_cast<float4*>(to + ch) =
                    make_float4(st.o[n][d][i] * unit_of, st.o[n][d][i + 2] * unit_of,
                                st.o[n][d + 1][i] * unit_of, st.o[n][d + 1][i + 2] * unit_of);
            }
        }
    __syncthreads();
    // The CTA's rows, then (S > 1) the cluster's: four channels to a thread.
    constexpr int kQuads = D / 4;
    for (int i = tid; i < R * kQuads; i += kThreads) {
        const int r = i / kQuads, d = i % kQuads * 4;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, part_m[w * R + r]);
        float l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = part_m[w * R + r];
            const float f = mw == -INFINITY ? 0.0f : ex2(mw - m);
            if (mw == -INFINITY) continue;
            l += f * part_l[w * R + r];
            const float4 y = *reinterpret_cast<const float4*>(part + (w * R + r) * kStride + d);
            o.x += f * y.x;
            o.y += f * y.y;
            o.z += f * y.z;
            o.w += f * y.w;
        }
        *reinterpret_cast<float4*>(mine + r * kStride + d) = o;
        if (d == 0) {
            mine_m[r] = m;
            mine_m[R + r] = l;
        }
    }
    if (S > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    for (int i = rank * kThreads + tid; i < rows * kQuads; i += S * kThreads) {
        const int r = i / kQuads, d = i % kQuads * 4;
        const uint32_t at_m = ptx::smem_u32(mine_m + r), at_o = ptx::smem_u32(mine + r * kStride + d);
        float m = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < S; ++s) m = fmaxf(m, ptx::ld_cluster(ptx::map_rank(at_m, s)));
        for (int s = 0; s < S; ++s) {
            const float ms = ptx::ld_cluster(ptx::map_rank(at_m, s));
            if (ms == -INFINITY) continue;
            const float f = ex2(ms - m);
            l += f * ptx::ld_cluster(ptx::map_rank(at_m + 4 * R, s));
            const float4 y = ptx::ld_cluster_v4(ptx::map_rank(at_o, s));
            o.x += f * y.x;
            o.y += f * y.y;
            o.z += f * y.z;
            o.w += f * y.w;
        }
        const bool none = m == -INFINITY;
        const float inv = none ? 0.0f : 1.0f / l;
        *reinterpret_cast<uint2*>(a.out + (row0 + r) * D + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (d == 0) a.lse[row0 + r] = none ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
    }
    if (S > 1) ptx::cluster_sync();  // (other CTAs may still read this one's rows)
}

template <int D, int NT>
size_t smem_bytes(int n_blocks) {
    constexpr int R = 8 * NT;
    return static_cast<size_t>((kWarps + 1) * R * (D + 4) + (kWarps + 1) * R * 2) * 4 +
           static_cast<size_t>(n_blocks) * 8;
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

template <int D, bool FP8, int NT>
int launch(const Args& a, int units, int sms, cudaStream_t stream) {
    const size_t smem = smem_bytes<D, NT>(a.n_blocks);
    const void* kernel = reinterpret_cast<const void*>(blocks_kernel<D, FP8, NT>);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
        return TREE_ATTN_ERR_CUDA;
    // CTAs of a cluster: as many as the SMs hold at once, while each warp has a tile.
    const int resident = NT == 1 ? 2 : 1;
    const long long tiles = static_cast<long long>(a.n_blocks < a.max_pages ? a.n_blocks : a.max_pages) *
                                (a.P / kTile) + (a.T + kTile - 1) / kTile;
    int S = 1;
    while (S < 8 && 2LL * S * units <= static_cast<long long>(resident) * sms &&
           tiles >= 2LL * S * kWarps)
        S *= 2;
    return rc_of(launch_cluster(blocks_kernel<D, FP8, NT>, dim3(static_cast<unsigned>(units) * S),
                                dim3(kThreads), smem, S, stream, a));
}

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" int tree_attn_verify_blocks(
    const uint16_t* q, const void* k_pages, const void* v_pages, const uint8_t* k_scales,
    const uint8_t* v_scales, const int32_t* block_table, int max_pages_per_seq,
    const int32_t* seq_lens, const int32_t* blocks, int n_blocks, const uint16_t* tree_k,
    const uint16_t* tree_v, const uint64_t* mask, int mask_stride, const int32_t* parents,
    int parents_stride, uint16_t* out, float* lse, int B, int Hq, int Hkv, int d, int T,
    int page_size, int num_pages, float softmax_scale, int32_t* status, void* stream) {
    if (B < 0 || Hkv < 1 || Hkv > 65535 || Hq < 1 || Hq % Hkv != 0 || (d != 64 && d != 128) ||
        T < 1 || T > TREE_ATTN_MAX_T || !page_size_ok(page_size) || max_pages_per_seq < 1 ||
        num_pages < 1 || static_cast<long long>(num_pages) * Hkv * page_size >= (1LL << 31) ||
        static_cast<long long>(max_pages_per_seq) * page_size >= (1LL << 31) || n_blocks < 0 ||
        n_blocks > 4096 || !std::isfinite(softmax_scale) ||
        (mask != nullptr && parents != nullptr) ||
        (mask != nullptr && mask_stride != 0 && mask_stride != T) ||
        (parents != nullptr && parents_stride != 0 && parents_stride != T) ||
        (k_scales == nullptr) != (v_scales == nullptr))
        return TREE_ATTN_ERR_SHAPE;
    const int G = Hq / Hkv;
    const int NT = G > 8 ? 2 : 1;
    const int row_blocks = (G + 8 * NT - 1) / (8 * NT);
    const long long units = static_cast<long long>(B) * Hkv * T * row_blocks;
    if (units * 8 >= (1LL << 31)) return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    if (!q || !k_pages || !v_pages || !block_table || !seq_lens || (n_blocks > 0 && !blocks) ||
        !tree_k || !tree_v || (!mask && !parents) || !out || !lse)
        return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(q, 16) || !ptr_aligned(k_pages, 16) || !ptr_aligned(v_pages, 16) ||
        !ptr_aligned(tree_k, 16) || !ptr_aligned(tree_v, 16) || !ptr_aligned(out, 16) ||
        !ptr_aligned(block_table, 4) || !ptr_aligned(seq_lens, 4) || !ptr_aligned(blocks, 4) ||
        !ptr_aligned(lse, 4) || !ptr_aligned(mask, 8) || !ptr_aligned(parents, 4) ||
        !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return TREE_ATTN_ERR_CUDA;
    Args a;
    a.q = q;
    a.kv[0] = k_pages;
    a.kv[1] = v_pages;
    a.scales[0] = k_scales;
    a.scales[1] = v_scales;
    a.table = block_table;
    a.lens = seq_lens;
    a.blocks = blocks;
    a.tree[0] = tree_k;
    a.tree[1] = tree_v;
    a.mask = mask;
    a.parents = parents;
    a.out = out;
    a.lse = lse;
    a.n_blocks = n_blocks;
    a.max_pages = max_pages_per_seq;
    a.mask_stride = mask_stride;
    a.parents_stride = parents_stride;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.T = T;
    a.P = page_size;
    a.num_pages = num_pages;
    a.row_blocks = row_blocks;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.status = status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int u = static_cast<int>(units);
    const bool f = k_scales != nullptr;
    if (d == 128) {
        if (NT == 1) return f ? launch<128, true, 1>(a, u, sms, s) : launch<128, false, 1>(a, u, sms, s);
        return f ? launch<128, true, 2>(a, u, sms, s) : launch<128, false, 2>(a, u, sms, s);
    }
    if (NT == 1) return f ? launch<64, true, 1>(a, u, sms, s) : launch<64, false, 1>(a, u, sms, s);
    return f ? launch<64, true, 2>(a, u, sms, s) : launch<64, false, 2>(a, u, sms, s);
}
