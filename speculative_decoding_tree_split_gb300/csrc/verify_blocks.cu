// verify_blocks.cu -- split tree attention over selected pages of a bf16 or 8-bit
// cache (one token per sequence: sparse decoding).
//
// Every (sequence, token, KV head) has its own list of pages.  Tokens of a sequence
// share most of theirs, so a unit of work is up to 8 or 16 query rows -- the G heads of
// one or several tokens -- and the union of their lists, each page with the tokens that
// list it; a page is read once and its scores hidden from the other tokens.  The work
// is reading pages.  A unit is split over the CTAs of a cluster and the warps of a CTA,
// 16 keys to a tile; each warp keeps running maxima, sums and accumulators of its own,
// which the CTA joins through shared memory and the cluster through one another's, so
// there is one launch and no workspace.
//
// K and V tiles come by asynchronous copies into a ring of each warp's own, K and V
// apart, so that the next ones are on their way while one is worked on and no register
// waits for them.  With S^T = K Q^T and O^T = V^T P^T the keys (channels) are the 16-row
// side and the query rows the 8-column side, so no half of a tile is padding for 8 rows,
// and since the order of channels within the product is free, it is chosen so that 32
// (K) or 16 (V) contiguous bytes of a row are a lane's operands.  V's pairs of keys are
// put together by byte permutes, P turns from result to operand by movmatrix.
//
// Measured, 64 sequences of 512 to 16384 tokens, 32 heads on 8 of 128, 32 pages of 64
// tokens: one token bf16 82 us (5.9 TB/s), 8-bit 53 (4.6 TB/s); four tokens with lists of
// their own, bf16 150 (5.6 TB/s), 8-bit, 428 MB, 98 (4.4 TB/s).  The bf16 form is bound by
// memory, the 8-bit one by the rate of instructions: 475 to a tile of 16 keys and 16 rows,
// most of them conversions of codes, at 2.1 a clock of an SM, whose registers hold two CTAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/tree_attn.h"
#include "cluster.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "layout.h"
#include "mma_sync.cuh"
#include "ptx.cuh"
#include "ptx_serving.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kResident = 2;  // CTAs of an SM: 128 registers, and half of the shared memory
constexpr int kTile = 16;        // keys
constexpr int kWindow = 4096;    // pages of a sequence that are marked at a time
constexpr int kMostEntries = 4096;
constexpr int kFixed = 8;
// References.  With a bf16 cache a row's is the largest score that it had when it last
// moved, which it does where a score exceeds it by more than kMove binades.  With an 8-bit
// one the scale of a key's value joins its exponent, e = x + s, p = 2^(e - reference): o
// sums p times the value's codes, the row's sum takes p 2^-s.  So a large scale costs only
// rows that see it, and those no more than their own largest p max|v| says.  p goes to
// the product as fp16 and may reach 2^kMost; a new reference leaves the largest at
// 2^kFresh, or as near as fp16 does not tell apart: a key that has most of its row is then
// rounded by less than 2^-15, not 2^-12.  (A reference is a multiple of 1 / kGrid, so that
// s less it is exact.)
constexpr float kMove = 8.0f;
constexpr float kMost = 15.0f, kFresh = 7.0f, kGrid = 16384.0f;
constexpr float kLeast = 1.17549435e-38f;  // of a score unit: never 0, which would lose -inf
constexpr float kLow = -3.0e38f; // a reference before the first key

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
    int tokens, groups;  // of a unit, and units of a sequence's tokens
    int B;
    bool longest_first;
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
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// 8-bit cache: exponents s of the value scales of a lane's two keys, and 2^-s.  (With s in
// [-56, 40] a p that fp32 does not hold takes less than 2^-70 from the row's sum, of which
// the largest p has 2^-33 or more.)
struct ValueScales {
    float s[2] = {0.0f, 0.0f}, inv[2] = {1.0f, 1.0f};
    __device__ __forceinline__ void set(int i, uint32_t byte) {
        s[i] = static_cast<float>(static_cast<int>(byte) - 127);
        inv[i] = __int_as_float(max(254 - static_cast<int>(byte), 0) << 23);
    }
};

// One warp's running state for NT * 8 query rows; a lane holds columns 2c and
// 2c + 1 of every column tile.  Scores x come in units that make a logarithm to base 2
// of them by a factor (> 0), a column's own (8-bit cache) or one for all.
template <int D, bool FP8, int NT>
struct State {
    float unit[FP8 ? NT : 1][FP8 ? 2 : 1];
    float m[NT][2];           // references, logarithms to base 2 (kLow: of no key yet)
    float l[NT][2];           // this lane's part of the sums
    float o[NT][D / 16][4];   // [column tile][channel tile]

    __device__ __forceinline__ float factor(int n, int i) const {
        return FP8 ? unit[FP8 ? n : 0][FP8 ? i : 0] : unit[0][0];
    }
    // Logarithms above the references.
    __device__ __forceinline__ void above(float (&y)[NT][4], const float (&x)[NT][4],
                                          const ValueScales& v) const {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[n][i] = fmaf(x[n][i], factor(n, i & 1),
                               FP8 ? v.s[i >> 1] - m[n][i & 1] : -m[n][i & 1]);
    }
};

// The multiple of 1 / kGrid nearest to t; t itself where fp32 has few finer steps or none.
__device__ __forceinline__ float on_grid(float t) {
    return fabsf(t) < 1024.0f ? rintf(t * kGrid) * (1.0f / kGrid) : t;
}

// Scores to probabilities (in place), summed; the references are moved where one is
// exceeded by too much.
template <int D, bool FP8, int NT>
__device__ __forceinline__ void exponents(State<D, FP8, NT>& st, float (&x)[NT][4],
                                          const ValueScales& v) {
    float y[NT][4];
    st.above(y, x, v);
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, y[n][i]);
    if (__any_sync(kFull, top > (FP8 ? kMost : kMove))) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float t = FP8 ? fmaxf(fmaf(x[n][i], st.factor(n, i), v.s[0]),
                                      fmaf(x[n][i + 2], st.factor(n, i), v.s[1]))
                              : fmaxf(x[n][i], x[n][i + 2]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    t = fmaxf(t, __shfl_xor_sync(kFull, t, off));
                t = fmaxf(FP8 ? on_grid(t) - kFresh : t * st.factor(n, i), st.m[n][i]);
                f[i] = ex2(st.m[n][i] - t);
                st.m[n][i] = t;
                st.l[n][i] *= f[i];
            }
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) st.o[n][d][i] *= f[i & 1];
        }
        st.above(y, x, v);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[n][i] = ex2(y[n][i]);
            st.l[n][i & 1] = FP8 ? fmaf(x[n][i], v.inv[i >> 1], st.l[n][i & 1])
                                 : st.l[n][i & 1] + x[n][i];
        }
}

// O^T += V^T P^T for one tile of channels: an accumulator that takes all, or (columns
// whose `mine` is false keep what they have) one apart that is added where it belongs.
template <bool CAREFUL, typename Mma>
__device__ __forceinline__ void add_tile(float (&o)[4], const bool (&mine)[2], Mma mma) {
    if (!CAREFUL) {
        mma(o);
    } else {
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma(y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (mine[i & 1]) o[i] += y[i];
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

// Queries in shared memory, 2-byte values: vector j (of D / 32) of lane c of a row, the
// four lanes' next to one another, rows 64 bytes apart beyond their length, so that the
// two rows that a quarter of a warp reads fall on different banks.
template <int D>
__device__ __forceinline__ int query_at(int row, int j, int c) {
    return row * (2 * D + 64) + j * 64 + c * 16;
}
template <int D>
__device__ __forceinline__ uint4 query(const uint8_t* q, int row, int j, int c) {
    return *reinterpret_cast<const uint4*>(q + query_at<D>(row, j, c));
}

// ---- tiles of 16 rows of RB bytes in shared memory, 16-byte chunks of a row moved
// about so that a warp's reads of operands meet no bank twice

// Where chunk ch of a row lies: for K a lane reads two next to one another, eight lanes
// two rows; for V one of each of four even rows.
template <int RB, bool V>
__device__ __forceinline__ int chunk_at(int row, int ch) {
    if (RB < 128) return row * RB + (V ? ch ^ ((row >> 1) & 3) : ch) * 16;
    const int turn = V ? (row >> 1 & 3) << 1 : row & 1;
    return row * RB + (ch & ~7) * 16 + ((ch & 7) ^ turn) * 16;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All of this thread's copies but the last N groups have arrived; then all lanes'.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();
}

// One warp copies a tile of rows next to one another, 512 bytes at a time.  Where a
// lane's chunk goes changes in few bits from one time to the next.
template <int RB, bool V>
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint8_t* src) {
    constexpr int kChunks = RB / 16;
    const int lane = threadIdx.x & 31;
    const int at = chunk_at<RB, V>(lane / kChunks, lane % kChunks);
    src += lane * 16;
#pragma unroll
    for (int i = 0; i < RB * kTile / 512; ++i) {
        // Row lane / kChunks + 32 / kChunks * i: what that adds to (row / 2) % 4.
        const int turn = !V || RB < 128 ? 0 : RB == 128 ? (i & 1) * 64 : (i & 3) * 32;
        copy16(dst + (at ^ turn) + i * 512, src + i * 512);
    }
}

// The same with row r from row(r).
template <int RB, bool V, typename Row>
__device__ __forceinline__ void copy_rows(uint32_t dst, Row row) {
    constexpr int kChunks = RB / 16;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kChunks * kTile / 32; ++i) {
        const int id = lane + 32 * i, r = id / kChunks, ch = id % kChunks;
        copy16(dst + chunk_at<RB, V>(r, ch), reinterpret_cast<const uint8_t*>(row(r)) + ch * 16);
    }
}

// S^T += K Q^T for 16 bf16 keys; the query operand in shared memory: [row][channels in
// the order of K's chunks].
template <int D, int NT>
__device__ __forceinline__ void scores_bf16(float (&x)[NT][4], uint32_t k, const uint8_t* q, int g,
                                            int c) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const int ch = j / 2 * 8 + 2 * c + (j & 1);
        const uint4 k0 = ptx::ld_shared_v4(k + chunk_at<2 * D, false>(g, ch));
        const uint4 k1 = ptx::ld_shared_v4(k + chunk_at<2 * D, false>(g + 8, ch));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 y = query<D>(q, n * 8 + g, j, c);
            ptx::mma_sync_bf16(x[n], k0.x, k1.x, k0.y, k1.y, y.x, y.y);
            ptx::mma_sync_bf16(x[n], k0.z, k1.z, k0.w, k1.w, y.z, y.w);
        }
    }
}

// A lane's 16 bytes of the values of rows 2c, 2c + 1, 2c + 8 and 2c + 9; those of keys
// that are not there are cleared: a probability of 0 times a value that is no number is
// no number.
template <int RB>
__device__ __forceinline__ void load_values(uint4 (&v)[4], uint32_t at, int ch, int c, int live) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 2 * c + (r & 1) + 8 * (r >> 1);
        v[r] = ptx::ld_shared_v4(at + chunk_at<RB, true>(row, ch));
    }
    if (live < kTile) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (2 * c + (r & 1) + 8 * (r >> 1) >= live) v[r] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// A pair of bf16 numbers with 0 for those that are infinite.
__device__ __forceinline__ uint32_t without_infinities(uint32_t pair) {
    if ((pair & 0x7fffu) == 0x7f80u) pair &= 0xffff0000u;
    if ((pair & 0x7fff0000u) == 0x7f800000u) pair &= 0xffffu;
    return pair;
}

// O^T += V^T P^T for 16 keys of bf16 values, the probabilities as two bf16 numbers: what one leaves out (2^-9) would be the largest error before the
// result is rounded, and the product is not what bounds the kernel.  SPREAD: a lane's
// channels are 8 of every 64, else D / 8 in a row.  CAREFUL: an infinite value goes with
// the first number alone, since the second may be 0 or below.
template <bool CAREFUL, bool SPREAD, int D, bool FP8, int NT>
__device__ __forceinline__ void add_values_bf16(State<D, FP8, NT>& st, const float (&p)[NT][4],
                                                uint32_t v_at, int live,
                                                const bool (&mine)[NT][2], int g, int c) {
    uint32_t b[NT][2][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float y0 = p[n][2 * h], y1 = p[n][2 * h + 1];
            const uint32_t hi = pack_bf16(y0, y1);
            const uint32_t lo =
                pack_bf16(y0 - __uint_as_float(hi << 16), y1 - __uint_as_float(hi & 0xffff0000u));
            b[n][0][h] = ptx::transpose8(hi);
            b[n][1][h] = ptx::transpose8(lo);
        }
    }
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
        uint4 v[4];
        load_values<2 * D>(v, v_at, SPREAD ? 8 * h + g : g * (D / 64) + h, c, live);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t k0 = word(v[0], w), k1 = word(v[1], w);
            const uint32_t k2 = word(v[2], w), k3 = word(v[3], w);
            const uint32_t a0 = __byte_perm(k0, k1, 0x5410), a1 = __byte_perm(k0, k1, 0x7632);
            const uint32_t a2 = __byte_perm(k2, k3, 0x5410), a3 = __byte_perm(k2, k3, 0x7632);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                add_tile<CAREFUL>(st.o[n][h * 4 + w], mine[n], [&](float (&o)[4]) {
                    ptx::mma_sync_bf16(o, a0, a1, a2, a3, b[n][0][0], b[n][0][1]);
                    if (CAREFUL)
                        ptx::mma_sync_bf16(o, without_infinities(a0), without_infinities(a1),
                                           without_infinities(a2), without_infinities(a3),
                                           b[n][1][0], b[n][1][1]);
                    else
                        ptx::mma_sync_bf16(o, a0, a1, a2, a3, b[n][1][0], b[n][1][1]);
                });
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
// Scores hidden from the columns of other tokens.
template <int NT>
__device__ __forceinline__ void hide_others(float (&x)[NT][4], const bool (&mine)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!mine[n][i & 1]) x[n][i] = -INFINITY;
}

// Whether some accumulator of the warp is no finite number.
template <int D, bool FP8, int NT>
__device__ __forceinline__ bool not_finite(const State<D, FP8, NT>& st) {
    float y = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) y = fmaf(st.o[n][d][i], 0.0f, y);
    return __any_sync(kFull, y != 0.0f);
}

// Exclusive prefix of v over the CTA; the sum in `total`.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int s = sums[w];
        before += w < warp ? s : 0;
        total += s;
    }
    return before + x - v;
}

// One page of a unit's list: its first row of the pools (for the unit's KV head), its
// committed tokens, and (from bit 8 on) the tokens of the unit that list it.
struct Entry {
    int row;
    uint32_t live_who;
};

template <int D, bool FP8, int NT>
struct Smem {
    static constexpr int R = 8 * NT;         // query rows
    static constexpr int kStride = D + 4;    // floats of a partial row
    static constexpr int RB = FP8 ? D : 2 * D;       // bytes of a cache row
    // K or V of a tile; 8-bit cache: behind K the scales of its keys and of their values.
    static constexpr int kSlot = kTile * RB + (FP8 ? 32 : 0);
    // Slots of a warp's ring: 8 and 12 KB (d = 128), which also hold a tile of tree tokens.
    static constexpr int kSlots = FP8 ? 4 : 3;
    union alignas(16) Warp {
        uint8_t ring[kSlots * kSlot];
        float rows[R][kStride];              // the warp's own, in the end
    };
    Warp warp[kWarps];
    float part_m[kWarps][R], part_l[kWarps][R];
    alignas(16) float mine[R][kStride];      // the CTA's own rows
    float mine_m[R], mine_l[R];
    float unit[R], inv[R];                   // 8-bit cache: a row's score unit, and its factor
    alignas(16) uint8_t q[FP8 ? 2 : 1][R * (2 * D + 64)];  // queries for the pages, and (8-bit) for the tree
    int8_t seen[R][TREE_ATTN_MAX_T];         // tree tokens that each token sees
    int n_seen[R];
    int sums[kWarps];
    alignas(16) Entry entries[1];            // [tokens * n_blocks]

    // Tokens that list a page, 16 bits each, and the pages' rows, while the list is made.
    __device__ __forceinline__ uint32_t* marks() {
        static_assert(sizeof(warp) >= kWindow * (2 + 4), "a window's marks and rows");
        static_assert(sizeof(Warp::ring) >= 2 * kTile * 2 * D, "a tile of tree tokens");
        return reinterpret_cast<uint32_t*>(&warp[0]);
    }
};

// What a warp has to know of its unit.
struct Unit {
    int b, hk, nt, per_token, rows, n_entries;
    int turn, step;  // of the tiles it takes
};

// One warp's tiles, its rows left in shared memory.  A value that is no finite number must
// not reach tokens that do not see it, but a product gives it to all, and an infinite one
// must not meet both parts of a probability.  So that the tiles need not look, the warp
// looks at what it has in the end: if that is not finite, it leaves nothing (false) and
// takes its tiles again, CAREFUL.
template <int D, bool FP8, int NT, bool CAREFUL>
__device__ __forceinline__ bool warp_rows(const Args& a, Smem<D, FP8, NT>& sm, const Unit& u) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const unsigned everyone = (1u << u.nt) - 1u;
    unsigned token[NT][2];  // of this lane's columns, as a bit
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = n * 8 + 2 * c + i;
            token[n][i] = r < u.rows ? 1u << (r / u.per_token) : 0u;
        }
    State<D, FP8, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (FP8) st.unit[FP8 ? n : 0][FP8 ? i : 0] = sm.unit[n * 8 + 2 * c + i];
    if (!FP8) st.unit[0][0] = fmaxf(fabsf(a.scale_log2), kLeast);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            st.m[n][i] = kLow;
            st.l[n][i] = 0.0f;
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][d][i] = 0.0f;
    }

    // ---- pages
    // Tile i is rows i % (P / 16) * 16 of page i / (P / 16); a warp takes every step-th,
    // step being a multiple of 8 and so of a page's tiles: the same rows of all its pages.
    const int per_page = a.P / kTile, shift = __ffs(per_page) - 1;
    const int tiles = u.n_entries << shift;
    const int off = (u.turn & (per_page - 1)) * kTile;
    const int e0 = u.turn >> shift, e_step = u.step >> shift;
    using Sm = Smem<D, FP8, NT>;
    constexpr int RB = Sm::RB;
    const uint32_t ring = ptx::smem_u32(sm.warp[warp].ring);
    // The next entry from e on whose tile has keys (others are passed over), and what it says.
    auto find = [&](int e, Entry& en) {
        for (; e < u.n_entries; e += e_step) {
            en = sm.entries[e];
            if (static_cast<int>(en.live_who & 255u) > off) break;
        }
        return e;
    };
    // The copies run ahead by the ring's slots: K of a tile, V of it, K of the next.
    Entry next;
    int ahead = find(e0, next);
    auto copy_next = [&](uint32_t slot, auto values) {
        constexpr bool V = decltype(values)::value;
        if (ahead < u.n_entries) {
            const int first = next.row + off;
            const uint8_t* base =
                static_cast<const uint8_t*>(a.kv[V ? 1 : 0]) + static_cast<size_t>(first) * RB;
            copy_tile<RB, V>(slot, base);
            if (FP8 && !V && lane < 2) copy16(slot + kTile * RB + 16 * lane, a.scales[lane] + first);
            if (V) ahead = find(ahead + e_step, next);
        }
        copies_commit();
    };
    using std::bool_constant;
#pragma unroll
    for (int i = 0; i < Sm::kSlots; i += 2) {
        copy_next(ring + i * Sm::kSlot, bool_constant<false>());
        if (i + 1 < Sm::kSlots) copy_next(ring + (i + 1) * Sm::kSlot, bool_constant<true>());
    }
    // What is kSlots further on than K: K again, or V.
    using AfterK = bool_constant<Sm::kSlots % 2 != 0>;
    using AfterV = bool_constant<Sm::kSlots % 2 == 0>;
    uint32_t slot = ring;
    // The slot's copies have arrived; it has been read and is filled again.
    auto arrive = [&] { copies_wait<Sm::kSlots - 1>(); };
    auto refill = [&](auto values) {
        __syncwarp();
        copy_next(slot, values);
        slot += Sm::kSlot;
        if (slot == ring + Sm::kSlots * Sm::kSlot) slot = ring;
    };
    Entry here;
    for (int e = find(e0, here); e < u.n_entries; e = find(e + e_step, here)) {
        const int live = min(static_cast<int>(here.live_who & 255u) - off, kTile);
        const unsigned seers = here.live_who >> 8;
        float x[NT][4];
        ValueScales vs;
        arrive();
        if (!FP8) {
            scores_bf16<D, NT>(x, slot, sm.q[0], g, c);
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {  // 16 codes of a lane
                const int ch = D / 64 * c + j;
                const uint4 k0 = ptx::ld_shared_v4(slot + chunk_at<RB, false>(g, ch));
                const uint4 k1 = ptx::ld_shared_v4(slot + chunk_at<RB, false>(g + 8, ch));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        f16x2_of_e4m3x4(word(k0, 2 * h + w), f[w][0], f[w][2]);
                        f16x2_of_e4m3x4(word(k1, 2 * h + w), f[w][1], f[w][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 y = query<D>(sm.q[0], n * 8 + g, 2 * j + h, c);
                        ptx::mma_sync_f16(x[n], f[0][0], f[0][1], f[0][2], f[0][3], y.x, y.y);
                        ptx::mma_sync_f16(x[n], f[1][0], f[1][1], f[1][2], f[1][3], y.z, y.w);
                    }
                }
            }
            const float f0 = scale_of(ld_shared_u8(slot + kTile * RB + g));
            const float f1 = scale_of(ld_shared_u8(slot + kTile * RB + g + 8));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] *= j < 2 ? f0 : f1;
            vs.set(0, ld_shared_u8(slot + kTile * RB + 16 + g));
            vs.set(1, ld_shared_u8(slot + kTile * RB + 16 + g + 8));
        }
        refill(AfterK());
        if (live < kTile) hide<NT>(x, live, g);
        bool mine[NT][2];
        if (CAREFUL || seers != everyone) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) mine[n][j] = (token[n][j] & seers) != 0;
            hide_others<NT>(x, mine);
        }
        exponents(st, x, vs);
        arrive();
        if (!FP8) {
            add_values_bf16<CAREFUL, true>(st, x, slot, live, mine, g, c);
        } else {
            uint32_t p[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                p[n][0] = ptx::transpose8(pack_f16(x[n][0], x[n][1]));
                p[n][1] = ptx::transpose8(pack_f16(x[n][2], x[n][3]));
            }
            uint4 v[4];
            if (D == 128) {
                load_values<RB>(v, slot, g, c, live);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 2 * c + (r & 1) + 8 * (r >> 1);
                    const uint2 y =
                        ld_shared_v2(slot + chunk_at<RB, true>(row, g >> 1) + (g & 1) * 8);
                    v[r] = row < live ? make_uint4(y.x, y.y, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
                }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t k0 = word(v[0], w), k1 = word(v[1], w);
                const uint32_t k2 = word(v[2], w), k3 = word(v[3], w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // channels 4w + 2h and the next
                    uint32_t a0, a1, a2, a3;
                    f16x2_of_e4m3x4(__byte_perm(k0, k1, h ? 0x7362 : 0x5140), a0, a1);
                    f16x2_of_e4m3x4(__byte_perm(k2, k3, h ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        add_tile<CAREFUL>(st.o[n][2 * w + h], mine[n], [&](float (&o)[4]) {
                            ptx::mma_sync_f16(o, a0, a1, a2, a3, p[n][0], p[n][1]);
                        });
                }
            }
        }
        refill(AfterV());
    }

    // ---- tree tokens (bf16 in either cache): tiles of one token each, behind the pages'
    {
        const size_t stride = static_cast<size_t>(a.Hkv) * D;
        const size_t base = (static_cast<size_t>(u.b) * a.T * a.Hkv + u.hk) * D;
        int turn = tiles;
        for (int t = 0; t < u.nt; ++t) {
            for (int i = 0; i < sm.n_seen[t]; i += kTile, ++turn) {
                if (turn % u.step != u.turn) continue;
                const int here = min(sm.n_seen[t] - i, kTile);
                auto from = [&](const uint16_t* p, int r) {
                    return p + base + sm.seen[t][i + min(r, here - 1)] * stride;
                };
                const uint32_t v_at = ring + kTile * 2 * D;
                __syncwarp();  // (the ring has been read)
                copy_rows<2 * D, false>(ring, [&](int r) { return from(a.tree[0], r); });
                copy_rows<2 * D, true>(v_at, [&](int r) { return from(a.tree[1], r); });
                copies_commit();
                copies_wait<0>();
                float x[NT][4];
                scores_bf16<D, NT>(x, ring, sm.q[FP8 ? 1 : 0], g, c);
                bool mine[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) mine[n][j] = (token[n][j] >> t & 1u) != 0;
                    if (FP8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[n][j] *= sm.inv[n * 8 + 2 * c + (j & 1)];
                    }
                }
                hide<NT>(x, here, g);
                hide_others<NT>(x, mine);
                exponents(st, x, ValueScales());
                // (the accumulators' order of channels)
                add_values_bf16<CAREFUL, !FP8>(st, x, v_at, here, mine, g, c);
            }
        }
    }
    if (!CAREFUL && not_finite(st)) return false;

    // ---- this warp's rows to shared memory, where its ring was
    copies_wait<0>();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float l = st.l[n][i];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);
            const int r = n * 8 + 2 * c + i;
            if (g == 0) {
                sm.part_m[warp][r] = st.m[n][i];
                sm.part_l[warp][r] = l;
            }
#pragma unroll
            for (int d = 0; d < D / 16; d += 2) {
                const int ch = FP8 ? channel_fp8<D>(d, g) : channel_bf16<D>(d, g);
                *reinterpret_cast<float4*>(&sm.warp[warp].rows[r][ch]) =
                    make_float4(st.o[n][d][i], st.o[n][d][i + 2], st.o[n][d + 1][i],
                                st.o[n][d + 1][i + 2]);
            }
        }
    return true;
}

template <int D, bool FP8, int NT>
__device__ __noinline__ void warp_rows_again(const Args& a, Smem<D, FP8, NT>& sm, const Unit& u) {
    warp_rows<D, FP8, NT, true>(a, sm, u);
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, kResident)
    blocks_kernel(const __grid_constant__ Args a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int R = 8 * NT;
    Smem<D, FP8, NT>& sm = *reinterpret_cast<Smem<D, FP8, NT>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    // Units in the order (sequence, KV head, tokens, rows of a wide group).
    int unit = blockIdx.x / S;
    const int rb = unit % a.row_blocks;
    unit /= a.row_blocks;
    const int t0 = unit % a.groups * a.tokens;
    unit /= a.groups;
    const int hk = unit % a.Hkv;
    int b = unit / a.Hkv;
    if (a.longest_first) b = by_length(a.lens, a.B, b, reinterpret_cast<int*>(sm.entries));
    const int G = a.Hq / a.Hkv;
    const int nt = min(a.tokens, a.T - t0);
    const int per_token = min(G - rb * R, R);  // rows
    const int rows = nt * per_token;
    // Row r: head rb * R + r % per_token of token t0 + r / per_token.
    auto row_of = [&](int r) {
        return (static_cast<size_t>(b) * a.T + t0 + r / per_token) * a.Hq +
               static_cast<size_t>(hk) * G + rb * R + r % per_token;
    };

    // ---- all that can be asked for at once: the sequence's length, this thread's part of
    // the lists, of the queries and of the tree
    const int n_listed = nt * a.n_blocks;
    auto listed = [&](int i) {  // entry i of the unit's lists, token by token
        const int t = i / a.n_blocks;
        return a.blocks[((static_cast<size_t>(b) * a.T + t0 + t) * a.Hkv + hk) * a.n_blocks + i -
                        t * a.n_blocks];
    };
    const int L_raw = a.lens[b];
    const int j_mine = tid < n_listed ? listed(tid) : -1;
    const int j_then = nt == 1 && tid + 1 < n_listed ? listed(tid + 1) : -1;
    constexpr int kVecs = D / 8;  // 16-byte vectors of a row, one to a lane
    constexpr int kTurns = (R * kVecs + kThreads - 1) / kThreads;
    uint4 q_mine[kTurns];
#pragma unroll
    for (int h = 0; h < kTurns; ++h) {
        const int r = (tid + h * kThreads) / kVecs;
        q_mine[h] = r < rows
                        ? *reinterpret_cast<const uint4*>(a.q + row_of(r) * D + tid % kVecs * 8)
                        : make_uint4(0u, 0u, 0u, 0u);
    }
    const int32_t* up = a.parents + static_cast<size_t>(b) * a.parents_stride;
    const int p0 = a.mask == nullptr && lane < a.T ? up[lane] : -1;
    const int p1 = a.mask == nullptr && lane + 32 < a.T ? up[lane + 32] : -1;

    // ---- the list of pages
    bool bad;
    const int L = clamp_seq_len(L_raw, a.P, a.max_pages, bad);
    if (bad && tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    const int nb = (L + a.P - 1) / a.P;
    const int32_t* table = a.table + static_cast<size_t>(b) * a.max_pages;
    // First row of logical page j of the sequence, -1 where there is none.
    auto page_row = [&](int j) {
        const int page = table[j];
        if (page >= 0 && page < a.num_pages) return (page * a.Hkv + hk) * a.P;  // (below 2^31)
        report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
        return -1;
    };
    auto entry = [&](int j, int row, unsigned who) {
        Entry e;
        e.row = max(row, 0);
        e.live_who = row < 0 ? 0u : static_cast<uint32_t>(min(a.P, L - j * a.P)) | who << 8;
        return e;
    };
    // One token whose list ascends (as it comes from the selection) is taken as it is.
    int n_entries = 0;
    bool as_is = nt == 1;
    if (as_is) {
        bool ascends = true;
        int n = 0;
        for (int i = tid; i < n_listed; i += kThreads) {
            const int j = i == tid ? j_mine : listed(i);
            const int then = i == tid ? j_then : i + 1 < n_listed ? listed(i + 1) : -1;
            ascends &= then < 0 || (j >= 0 && j < then);
            if (j < -1 || j >= nb) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            const bool ok = j >= 0 && j < nb;
            if (ok) sm.entries[i] = entry(j, page_row(j), 1u);
            n += ok;
        }
        as_is = __syncthreads_and(ascends);
        block_scan(n, sm.sums, n_entries);
    }
    if (!as_is) {
        n_entries = 0;
        uint32_t* marks = sm.marks();  // and behind them the pages' rows
        int* row_at = reinterpret_cast<int*>(marks + kWindow / 2);
        if (nb == 0) {  // (no window looks at the lists then)
            for (int i = tid; i < n_listed; i += kThreads)
                if (listed(i) != -1) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
        }
        for (int w0 = 0; w0 < nb; w0 += kWindow) {
            const int width = min(kWindow, nb - w0);
            __syncthreads();
            for (int i = tid; i < (width + 1) / 2; i += kThreads) marks[i] = 0;
            __syncthreads();
            for (int i = tid; i < n_listed; i += kThreads) {
                const int j = i == tid ? j_mine : listed(i);
                if (j < -1 || j >= nb) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                if (j >= w0 && j < w0 + width) {
                    const int at = j - w0;
                    atomicOr(marks + (at >> 1), 1u << (i / a.n_blocks + 16 * (at & 1)));
                    row_at[at] = page_row(j);  // (the same from all)
                }
            }
            __syncthreads();
            for (int i0 = 0; i0 < (width + 1) / 2; i0 += kThreads) {
                const int i = i0 + tid;
                const uint32_t m = i < (width + 1) / 2 ? marks[i] : 0u;
                const unsigned lo = m & 0xffffu, hi = m >> 16;
                int total;
                int at = n_entries + block_scan((lo != 0) + (hi != 0), sm.sums, total);
                if (lo != 0) sm.entries[at++] = entry(w0 + 2 * i, row_at[2 * i], lo);
                if (hi != 0) sm.entries[at] = entry(w0 + 2 * i + 1, row_at[2 * i + 1], hi);
                n_entries += total;
            }
        }
    }

    // ---- tree tokens that each token sees
    for (int t = warp; t < nt; t += kWarps) {
        uint64_t bits = 0;
        if (a.mask != nullptr) {
            bits = a.mask[static_cast<size_t>(b) * a.mask_stride + t0 + t];
            if (a.T < 64) bits &= (1ull << a.T) - 1ull;
        } else {
            if (p0 < -1 || (p0 >= lane && lane < a.T) || p1 < -1 ||
                (p1 >= lane + 32 && lane + 32 < a.T))
                report(a.status, TREE_ATTN_STATUS_BAD_PARENT);
            __syncwarp();
            int j = t0 + t;
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
                sm.seen[t][__popcll(bits & ((1ull << j) - 1ull))] = static_cast<int8_t>(j);
        }
        if (lane == 0) sm.n_seen[t] = __popcll(bits);
    }

    // ---- queries, as the product's second operand (8-bit cache: in fp16, scaled so that
    // the row's largest lies in [2^14, 2^15): exact down to 2^-28 of it, and to 2^-39 of
    // it below; and in bf16 for the tree)
#pragma unroll
    for (int h = 0; h < kTurns; ++h) {
        const int r = (tid + h * kThreads) / kVecs, i = tid % kVecs;
        if (r >= R) break;
        uint4 x = q_mine[h];
        if (a.scale_log2 < 0.0f) {  // score units are positive
            x.x ^= 0x80008000u;
            x.y ^= 0x80008000u;
            x.z ^= 0x80008000u;
            x.w ^= 0x80008000u;
        }
        // Vector i holds channels 8 i: in 64 channels 16 to a lane, or D / 4 to a lane.
        const int bf = query_at<D>(r, i / 8 * 2 + (i & 1), i % 8 / 2);
        if (FP8) {
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t y = word(x, w), lo = y & 0x7fffu, hi = (y >> 16) & 0x7fffu;
                top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            }
#pragma unroll
            for (int off = 1; off < kVecs; off <<= 1)
                top = max(top, __shfl_xor_sync(kFull, top, off));
            const int e = max(static_cast<int>(top >> 7) - 127 - 14, -112);
            const float inv = pow2(-e);
            uint32_t y[4];
#pragma unroll
            for (int w = 0; w < 4; ++w)
                y[w] = pack_f16(__uint_as_float(word(x, w) << 16) * inv,
                                __uint_as_float(word(x, w) & 0xffff0000u) * inv);
            *reinterpret_cast<uint4*>(sm.q[0] + query_at<D>(r, i % (D / 32), i / (D / 32))) =
                make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(sm.q[1] + bf) = x;
            if (i == 0) {
                sm.unit[r] = fmaxf(pow2(e) * fabsf(a.scale_log2), kLeast);
                sm.inv[r] = inv;
            }
        } else {
            *reinterpret_cast<uint4*>(sm.q[0] + bf) = x;
        }
    }

    Unit u;
    u.b = b;
    u.hk = hk;
    u.nt = nt;
    u.per_token = per_token;
    u.rows = rows;
    u.n_entries = n_entries;
    u.step = S * kWarps;
    u.turn = rank * kWarps + warp;
    __syncthreads();
    if (!warp_rows<D, FP8, NT, false>(a, sm, u)) warp_rows_again<D, FP8, NT>(a, sm, u);
    __syncthreads();
    // ---- the CTA's rows, and (S > 1) the cluster's: four channels to a thread
    constexpr int kQuads = D / 4;
    auto write = [&](int r, int d, float m, float l, const float4& o) {
        const bool none = l == 0.0f;  // no key at all
        const float inv = none ? 0.0f : 1.0f / l;
        const size_t row = row_of(r);
        *reinterpret_cast<uint2*>(a.out + row * D + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (d == 0) a.lse[row] = none ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
    };
    for (int i = tid; i < rows * kQuads; i += kThreads) {
        const int r = i / kQuads, d = i % kQuads * 4;
        float m = kLow;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.part_m[w][r]);
        float l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(sm.part_m[w][r] - m);
            l += f * sm.part_l[w][r];
            const float4 y = *reinterpret_cast<const float4*>(&sm.warp[w].rows[r][d]);
            o.x += f * y.x;
            o.y += f * y.y;
            o.z += f * y.z;
            o.w += f * y.w;
        }
        if (S == 1) {
            write(r, d, m, l, o);
        } else {
            *reinterpret_cast<float4*>(&sm.mine[r][d]) = o;
            if (d == 0) {
                sm.mine_m[r] = m;
                sm.mine_l[r] = l;
            }
        }
    }
    if (S == 1) return;
    ptx::cluster_sync();
    for (int i = rank * kThreads + tid; i < rows * kQuads; i += S * kThreads) {
        const int r = i / kQuads, d = i % kQuads * 4;
        const uint32_t at_m = ptx::smem_u32(&sm.mine_m[r]), at_l = ptx::smem_u32(&sm.mine_l[r]);
        const uint32_t at_o = ptx::smem_u32(&sm.mine[r][d]);
        float m = kLow, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s0 = 0; s0 < S; s0 += 4) {  // (four CTAs' at a time: one round trip)
            float ms[4], ls[4];
            float4 y[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t from = min(s0 + s, S - 1);
                ms[s] = ptx::ld_cluster(ptx::map_rank(at_m, from));
                ls[s] = ptx::ld_cluster(ptx::map_rank(at_l, from));
                y[s] = ptx::ld_cluster_v4(ptx::map_rank(at_o, from));
            }
            float top = m;
#pragma unroll
            for (int s = 0; s < 4; ++s) top = fmaxf(top, ms[s]);
            const float f0 = ex2(m - top);
            m = top;
            l *= f0;
            o.x *= f0;
            o.y *= f0;
            o.z *= f0;
            o.w *= f0;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s0 + s >= S) break;
                const float f = ex2(ms[s] - top);
                l += f * ls[s];
                o.x += f * y[s].x;
                o.y += f * y[s].y;
                o.z += f * y[s].z;
                o.w += f * y[s].w;
            }
        }
        write(r, d, m, l, o);
    }
    ptx::cluster_sync();  // (other CTAs may still read this one's rows)
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

template <int D, bool FP8, int NT>
int launch(Args a, long long units, int dev, int sms, cudaStream_t stream) {
    const size_t smem = sizeof(Smem<D, FP8, NT>) + (kThreads + 1) * sizeof(int) +
                        static_cast<size_t>(a.tokens) * a.n_blocks * sizeof(Entry);
    const auto kernel = blocks_kernel<D, FP8, NT>;
    static std::atomic<unsigned long long> ready{0};
    if (!opt_in(reinterpret_cast<const void*>(kernel), dev, ready, true)) return TREE_ATTN_ERR_CUDA;
    // CTAs of a cluster: those that take the least time, a CTA taking as long as a warp's
    // tiles and kFixed tiles' worth of beginning and end, and an SM with c of them c times
    // 0.62 of that (measured: two go on beside each other at 1.6 times the pace of one).
    const long long most = a.n_blocks < a.max_pages ? a.n_blocks : a.max_pages;
    const long long tiles = most * (a.P / kTile) * (a.tokens + 1) / 2 + a.tokens;
    int S = 1;
    long long best = -1;
    for (int s = 1; s <= 16; s *= 2) {
        const long long on_sm = (units * s + sms - 1) / sms;
        const long long each = (tiles + s * kWarps - 1) / (s * kWarps) + kFixed;
        const long long cost = each * (on_sm == 1 ? 100 : 62 * on_sm);
        if (best < 0 || cost < best) {
            best = cost;
            S = s;
        }
    }
    a.longest_first = a.B > 1 && a.B <= kThreads && units * S > kResident * sms;
    return rc_of(launch_cluster(kernel, dim3(static_cast<unsigned>(units * S)),
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
        n_blocks > kMostEntries || !std::isfinite(softmax_scale) ||
        (mask != nullptr && parents != nullptr) ||
        (mask != nullptr && mask_stride != 0 && mask_stride != T) ||
        (parents != nullptr && parents_stride != 0 && parents_stride != T) ||
        (k_scales == nullptr) != (v_scales == nullptr))
        return TREE_ATTN_ERR_SHAPE;
    const int G = Hq / Hkv;
    // Rows of a unit: 8 where that is all there are, else 16; tokens that fill them.
    const int NT = T * G > 8 ? 2 : 1;
    const int R = 8 * NT;
    const int row_blocks = (G + R - 1) / R;
    int tokens = G >= R ? 1 : R / G;
    if (tokens > T) tokens = T;
    while (tokens > 1 && tokens * n_blocks > kMostEntries) --tokens;
    const int groups = (T + tokens - 1) / tokens;
    const long long units = static_cast<long long>(B) * Hkv * groups * row_blocks;
    if (units * 16 >= (1LL << 31)) return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    if (!q || !k_pages || !v_pages || !block_table || !seq_lens || (n_blocks > 0 && !blocks) ||
        !tree_k || !tree_v || (!mask && !parents) || !out || !lse)
        return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(q, 16) || !ptr_aligned(k_pages, 16) || !ptr_aligned(v_pages, 16) ||
        !ptr_aligned(tree_k, 16) || !ptr_aligned(tree_v, 16) || !ptr_aligned(out, 16) ||
        !ptr_aligned(block_table, 4) || !ptr_aligned(seq_lens, 4) || !ptr_aligned(blocks, 4) ||
        !ptr_aligned(k_scales, 16) || !ptr_aligned(v_scales, 16) || !ptr_aligned(lse, 4) ||
        !ptr_aligned(mask, 8) || !ptr_aligned(parents, 4) ||
        !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    const int sms = sms_of(dev);
    if (sms == 0) return TREE_ATTN_ERR_CUDA;
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
    a.B = B;
    a.tokens = tokens;
    a.groups = groups;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.status = status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f = k_scales != nullptr;
    if (d == 128) {
        if (NT == 1) return f ? launch<128, true, 1>(a, units, dev, sms, s) : launch<128, false, 1>(a, units, dev, sms, s);
        return f ? launch<128, true, 2>(a, units, dev, sms, s) : launch<128, false, 2>(a, units, dev, sms, s);
    }
    if (NT == 1) return f ? launch<64, true, 1>(a, units, dev, sms, s) : launch<64, false, 1>(a, units, dev, sms, s);
    return f ? launch<64, true, 2>(a, units, dev, sms, s) : launch<64, false, 2>(a, units, dev, sms, s);
}
