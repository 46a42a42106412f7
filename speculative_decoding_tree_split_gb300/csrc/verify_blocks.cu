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
// K and V go from memory straight into the registers of the product: with
// S^T = K Q^T and O^T = V^T P^T the keys (channels) are the 16-row side and the
// query rows the 8-column side, so no half of a tile is padding for 8 rows, and
// since the order of channels within the product is free, it is chosen so that 32 (K)
// or 16 (V) contiguous bytes of a row are a lane's operands.  V's pairs of keys are put
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
constexpr int kTile = 16;        // keys
constexpr int kWindow = 8192;    // pages of a sequence that are marked at a time
constexpr int kMostEntries = 4096;
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
    int tokens, groups;  // of a unit, and units of a sequence's tokens
    bool wide;           // K's rows begin on 32-byte boundaries
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

// O^T += V^T P^T for one tile of channels: an accumulator that takes all, or (columns
// whose `mine` is false keep what they have) one apart that is added where it belongs.
template <typename Mma>
__device__ __forceinline__ void add_tile(float (&o)[4], const bool (&mine)[2], bool careful,
                                         Mma mma) {
    if (!careful) {
        mma(o);
    } else {
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma(y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (mine[i & 1]) o[i] += y[i];
    }
}

// O^T += V^T P^T for 16 keys of bf16 values, the probabilities (times f) as two
// bf16 numbers: what one leaves out (2^-9) would be the largest error before the
// result is rounded, and the product is not what bounds the kernel.
template <int D, int NT>
__device__ __forceinline__ void add_values_bf16(State<D, NT>& st, const float (&p)[NT][4],
                                                const uint4 (&v)[4][D / 64], float f,
                                                const bool (&mine)[NT][2], bool careful) {
    uint32_t b[NT][2][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float y0 = p[n][2 * h] * f, y1 = p[n][2 * h + 1] * f;
            const uint32_t hi = pack_bf16(y0, y1);
            const uint32_t lo =
                pack_bf16(y0 - __uint_as_float(hi << 16), y1 - __uint_as_float(hi & 0xffff0000u));
            b[n][0][h] = ptx::transpose8(hi);
            b[n][1][h] = ptx::transpose8(lo);
        }
    }
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t k0 = word(v[0][h], w), k1 = word(v[1][h], w);
            const uint32_t k2 = word(v[2][h], w), k3 = word(v[3][h], w);
            const uint32_t a0 = __byte_perm(k0, k1, 0x5410), a1 = __byte_perm(k0, k1, 0x7632);
            const uint32_t a2 = __byte_perm(k2, k3, 0x5410), a3 = __byte_perm(k2, k3, 0x7632);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                add_tile(st.o[n][h * 4 + w], mine[n], careful, [&](float (&o)[4]) {
                    ptx::mma_sync_bf16(o, a0, a1, a2, a3, b[n][0][0], b[n][0][1]);
                    ptx::mma_sync_bf16(o, a0, a1, a2, a3, b[n][1][0], b[n][1][1]);
                });
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

// 32 bytes of a row (`wide`: on a 32-byte boundary).
__device__ __forceinline__ void load32(uint4& lo, uint4& hi, const void* p, bool wide) {
    if (wide) {
        asm volatile(
            "ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z),
              "=r"(hi.w)
            : "l"(p));
    } else {
        lo = ptx::ld_stream(p);
        hi = ptx::ld_stream(static_cast<const uint8_t*>(p) + 16);
    }
}

// 16 bf16 keys: the lane's vectors of rows g and g + 8 (16 channels of every 64), and
// of the values of rows 2c, 2c + 1, 2c + 8, 2c + 9, by a function from row to address.
template <int D, typename Row>
__device__ __forceinline__ void load_keys_bf16(uint4 (&k)[2][D / 32], Row row, int g, int c,
                                               bool wide) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            load32(k[r][2 * j], k[r][2 * j + 1], row(g + 8 * r) + j * 64 + c * 16, wide);
}
template <int D, typename Row>
__device__ __forceinline__ void load_values_bf16(uint4 (&v)[4][D / 64], Row row, int g, int c) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            v[r][h] = ptx::ld_stream(row(2 * c + (r & 1) + 8 * (r >> 1)) + h * 64 + g * 8);
}

// The query operand in shared memory: [row][channels in the order of K's vectors].
template <int D, int NT>
__device__ __forceinline__ void scores_bf16(float (&x)[NT][4], const uint4 (&k)[2][D / 32],
                                            const uint8_t* q, int g, int c) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const uint4 y = query<D>(q, n * 8 + g, j, c);
            ptx::mma_sync_bf16(x[n], k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y, y.x, y.y);
            ptx::mma_sync_bf16(x[n], k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w, y.z, y.w);
        }
    }
}

// Keys past `live` seen by nobody.
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

// Whether some value of the tile is no finite number.
template <bool FP8, int N>
__device__ __forceinline__ bool not_finite(const uint4 (&v)[4][N]) {
    uint32_t bad = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int h = 0; h < N; ++h)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t x = word(v[r][h], w);
                bad |= FP8 ? ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u
                           : ((x & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
            }
    return __any_sync(kFull, bad != 0);
}

// Exclusive prefix of v over the CTA; the sum in `total`.
template <int W>
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
    for (int w = 0; w < W; ++w) {
        const int s = sums[w];
        before += w < warp ? s : 0;
        total += s;
    }
    return before + x - v;
}

// Warps of a CTA and CTAs of an SM: as many registers as two column tiles need leave
// room for twelve warps, one for sixteen.
template <int NT>
struct Shape {
    static constexpr int kWarps = NT == 1 ? 8 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kResident = NT == 1 ? 2 : 3;
};

// One page of a unit's list: its row of the pools, its committed tokens, and (from
// bit 8 on) the tokens of the unit that list it.
struct Entry {
    int page;
    uint32_t live_who;
};

template <int D, int NT>
struct Smem {
    static constexpr int kWarps = Shape<NT>::kWarps;
    static constexpr int R = 8 * NT;         // query rows
    static constexpr int kStride = D + 4;    // floats of a partial row
    float part[kWarps][R][kStride];
    float part_m[kWarps][R], part_l[kWarps][R];
    float mine[R][kStride];                  // the CTA's own rows
    float mine_m[R], mine_l[R];
    float unit[R];                           // of a row's scores
    uint8_t q[2][R * (2 * D + 64)];          // queries for the pages, and (8-bit) for the tree
    int8_t seen[R][TREE_ATTN_MAX_T];         // tree tokens that each token sees
    int n_seen[R];
    int sums[kWarps];
    Entry entries[1];                        // [tokens * n_blocks]

    // Tokens that list a page, 16 bits each, while the list is made (`part` is used last).
    __device__ __forceinline__ uint32_t* marks() {
        static_assert(sizeof(part) >= kWindow * 2, "a window's marks");
        return reinterpret_cast<uint32_t*>(&part[0][0][0]);
    }
};

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(Shape<NT>::kThreads, Shape<NT>::kResident)
    blocks_kernel(const Args a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kWarps = Shape<NT>::kWarps, kThreads = Shape<NT>::kThreads, R = 8 * NT;
    Smem<D, NT>& sm = *reinterpret_cast<Smem<D, NT>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int S = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    // Units in the order (sequence, KV head, tokens, rows of a wide group).
    int unit = blockIdx.x / S;
    const int rb = unit % a.row_blocks;
    unit /= a.row_blocks;
    const int t0 = unit % a.groups * a.tokens;
    unit /= a.groups;
    const int hk = unit % a.Hkv, b = unit / a.Hkv;
    const int G = a.Hq / a.Hkv;
    const int nt = min(a.tokens, a.T - t0);
    const int per_token = min(G - rb * R, R);  // rows
    const int rows = nt * per_token;
    const unsigned everyone = (1u << nt) - 1u;
    // Row r: head rb * R + r % per_token of token t0 + r / per_token.
    auto row_of = [&](int r) {
        return (static_cast<size_t>(b) * a.T + t0 + r / per_token) * a.Hq +
               static_cast<size_t>(hk) * G + rb * R + r % per_token;
    };

    // ---- the list of pages
    bool bad;
    const int L = clamp_seq_len(a.lens[b], a.P, a.max_pages, bad);
    if (bad && tid == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    const int nb = (L + a.P - 1) / a.P;
    const int32_t* table = a.table + static_cast<size_t>(b) * a.max_pages;
    auto list_of = [&](int t) {
        return a.blocks +
               ((static_cast<size_t>(b) * a.T + t0 + t) * a.Hkv + hk) * a.n_blocks;
    };
    auto entry = [&](int j, unsigned who) {
        Entry e;
        e.page = table[j];
        if (e.page < 0 || e.page >= a.num_pages) {
            report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            e.page = 0;
            who = 0;
        }
        e.live_who = static_cast<uint32_t>(who == 0 ? 0 : min(a.P, L - j * a.P)) | who << 8;
        return e;
    };
    // One token whose list ascends (as it comes from the selection) is taken as it is.
    int n_entries = 0;
    bool as_is = nt == 1;
    if (as_is) {
        const int32_t* list = list_of(0);
        bool ascends = true;
        int n = 0;
        for (int i = tid; i < a.n_blocks; i += kThreads) {
            const int j = list[i], then = i + 1 < a.n_blocks ? list[i + 1] : -1;
            ascends &= then < 0 || (j >= 0 && j < then);
            if (j < -1 || j >= nb) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            const bool ok = j >= 0 && j < nb;
            if (ok) sm.entries[i] = entry(j, 1u);
            n += ok;
        }
        as_is = __syncthreads_and(ascends);
        block_scan<kWarps>(n, sm.sums, n_entries);
    }
    if (!as_is) {
        n_entries = 0;
        for (int w0 = 0; w0 < nb; w0 += kWindow) {
            const int width = min(kWindow, nb - w0);
            uint32_t* marks = sm.marks();
            __syncthreads();
            for (int i = tid; i < (width + 1) / 2; i += kThreads) marks[i] = 0;
            __syncthreads();
            for (int t = 0; t < nt; ++t) {
                const int32_t* list = list_of(t);
                for (int i = tid; i < a.n_blocks; i += kThreads) {
                    const int j = list[i];
                    if (j < -1 || j >= nb) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                    if (j >= w0 && j < w0 + width)
                        atomicOr(marks + ((j - w0) >> 1), 1u << (t + 16 * ((j - w0) & 1)));
                }
            }
            __syncthreads();
            for (int i0 = 0; i0 < (width + 1) / 2; i0 += kThreads) {
                const uint32_t m = i0 + tid < (width + 1) / 2 ? marks[i0 + tid] : 0u;
                const unsigned lo = m & 0xffffu, hi = m >> 16;
                int total;
                int at = n_entries + block_scan<kWarps>((lo != 0) + (hi != 0), sm.sums, total);
                const int j = w0 + 2 * (i0 + tid);
                if (lo != 0) sm.entries[at++] = entry(j, lo);
                if (hi != 0) sm.entries[at] = entry(j + 1, hi);
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
            const int32_t* up = a.parents + static_cast<size_t>(b) * a.parents_stride;
            const int p0 = lane < a.T ? up[lane] : -1, p1 = lane + 32 < a.T ? up[lane + 32] : -1;
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
    constexpr int kVecs = D / 8;  // 16-byte vectors of a row, one to a lane
    for (int r = tid / kVecs; r < R; r += kThreads / kVecs) {
        const int i = tid % kVecs;
        const uint4 x = r < rows ? *reinterpret_cast<const uint4*>(a.q + row_of(r) * D + i * 8)
                                 : make_uint4(0u, 0u, 0u, 0u);
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
            if (i == 0) sm.unit[r] = pow2(e) * a.scale_log2;
        } else {
            *reinterpret_cast<uint4*>(sm.q[0] + bf) = x;
        }
    }

    State<D, NT> st;
    unsigned token[NT][2];  // of this lane's columns, as a bit
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            st.m[n][i] = -INFINITY;
            st.l[n][i] = 0.0f;
            const int r = n * 8 + 2 * c + i;
            token[n][i] = r < rows ? 1u << (r / per_token) : 0u;
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][d][i] = 0.0f;
    }
    int sref = kNoScale;  // 8-bit cache: accumulators are in units of 2^(sref - kLift)
    __syncthreads();

    // ---- pages
    const int per_page = a.P / kTile, shift = __ffs(per_page) - 1;
    const int tiles = n_entries << shift;
    const int step = S * kWarps;
    const int w0 = rank * kWarps + warp;
    // Tile i: its first row in the pools, its keys, and who sees them.
    int live = 0, at = 0;
    unsigned who = 0;
    size_t first = 0;
    auto next = [&](int from) {
        live = 0;
        for (at = from; at < tiles; at += step) {
            const Entry e = sm.entries[at >> shift];
            const int off = (at & (per_page - 1)) * kTile;
            live = min(max(static_cast<int>(e.live_who & 255u) - off, 0), kTile);
            who = e.live_who >> 8;
            first = (static_cast<size_t>(e.page) * a.Hkv + hk) * a.P + off;
            if (live > 0) break;  // (tiles without keys are passed over)
        }
    };
    next(w0);
    if (!FP8) {
        uint4 k[2][D / 32], v[4][D / 64];
        auto load_k = [&] {
            const uint16_t* base = static_cast<const uint16_t*>(a.kv[0]) + first * D;
            load_keys_bf16<D>(k, [&](int r) { return base + r * D; }, g, c, a.wide);
        };
        auto load_v = [&] {
            const uint16_t* base = static_cast<const uint16_t*>(a.kv[1]) + first * D;
            load_values_bf16<D>(v, [&](int r) { return base + r * D; }, g, c);
        };
        if (live > 0) {
            load_k();
            load_v();
        }
        while (live > 0) {
            float x[NT][4];
            scores_bf16<D, NT>(x, k, sm.q[0], g, c);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] *= a.scale_log2;
            const int now = live;
            const unsigned seers = who;
            next(at + step);
            if (live > 0) load_k();
            if (now < kTile) {
                hide<NT>(x, now, g);
                clear_values(v, now, c);
            }
            bool mine[NT][2], careful = false;
            if (seers != everyone) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) mine[n][i] = (token[n][i] & seers) != 0;
                hide_others<NT>(x, mine);
                careful = not_finite<false>(v);
            }
            follow(st, x);
            exponents(st, x);
            add_values_bf16<D, NT>(st, x, v, 1.0f, mine, careful);
            if (live > 0) load_v();
        }
    } else {
        constexpr int NC = D / 64;  // 16-byte vectors of a lane
        uint4 k[2][NC];
        uint4 v[4][1];
        uint32_t s[2][2];  // [K, V] scale bytes of keys g and g + 8
        auto load_k = [&] {
            const uint8_t* base = static_cast<const uint8_t*>(a.kv[0]) + first * D + c * (D / 4);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (D == 128)
                    load32(k[r][0], k[r][NC - 1], base + (g + 8 * r) * D, a.wide);
                else
                    k[r][0] = ptx::ld_stream(base + (g + 8 * r) * D);
                s[0][r] = a.scales[0][first + g + 8 * r];
            }
        };
        auto load_v = [&] {
            const uint8_t* base = static_cast<const uint8_t*>(a.kv[1]) + first * D + g * (D / 8);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint8_t* p = base + (2 * c + (r & 1) + 8 * (r >> 1)) * D;
                if (D == 128) {
                    v[r][0] = ptx::ld_stream(p);
                } else {
                    const uint2 y = ptx::ld_stream8(p);
                    v[r][0] = make_uint4(y.x, y.y, 0u, 0u);
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) s[1][r] = a.scales[1][first + g + 8 * r];
        };
        float rf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) rf[n][i] = sm.unit[n * 8 + 2 * c + i];
        if (live > 0) {
            load_k();
            load_v();
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
                for (int h = 0; h < 2; ++h) {  // eight codes of a lane
                    uint32_t f[2][4];
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        f16x2_of_e4m3x4(word(k[0][j], 2 * h + w), f[w][0], f[w][2]);
                        f16x2_of_e4m3x4(word(k[1][j], 2 * h + w), f[w][1], f[w][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 y = query<D>(sm.q[0], n * 8 + g, 2 * j + h, c);
                        ptx::mma_sync_f16(x[n], f[0][0], f[0][1], f[0][2], f[0][3], y.x, y.y);
                        ptx::mma_sync_f16(x[n], f[1][0], f[1][1], f[1][2], f[1][3], y.z, y.w);
                    }
                }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] = x[n][j] * scale_of(s[0][j >> 1]) * rf[n][j & 1];
            const int now = live;
            const unsigned seers = who;
            next(at + step);
            if (live > 0) load_k();
            int sv[2] = {static_cast<int>(s[1][0]) - 127, static_cast<int>(s[1][1]) - 127};
            if (now < kTile) {
                hide<NT>(x, now, g);
                if (g >= now) sv[0] = kNoScale;
                if (g + 8 >= now) sv[1] = kNoScale;
                clear_values(v, now, c);
            }
            bool mine[NT][2], careful = false;
            if (seers != everyone) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) mine[n][i] = (token[n][i] & seers) != 0;
                hide_others<NT>(x, mine);
                careful = not_finite<true>(v);
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
            uint32_t p[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    p[n][h] = ptx::transpose8(
                        pack_f16(x[n][2 * h] * pf[h], x[n][2 * h + 1] * pf[h]));
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t k0 = word(v[0][0], w), k1 = word(v[1][0], w);
                const uint32_t k2 = word(v[2][0], w), k3 = word(v[3][0], w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // channels 4w + 2h and the next
                    uint32_t a0, a1, a2, a3;
                    f16x2_of_e4m3x4(__byte_perm(k0, k1, h ? 0x7362 : 0x5140), a0, a1);
                    f16x2_of_e4m3x4(__byte_perm(k2, k3, h ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        add_tile(st.o[n][2 * w + h], mine[n], careful, [&](float (&o)[4]) {
                            ptx::mma_sync_f16(o, a0, a1, a2, a3, p[n][0], p[n][1]);
                        });
                }
            }
            if (live > 0) load_v();
        }
    }

    // ---- tree tokens (bf16 in either cache): tiles of one token each, behind the pages'
    {
        const size_t stride = static_cast<size_t>(a.Hkv) * D;
        const size_t base = (static_cast<size_t>(b) * a.T * a.Hkv + hk) * D;
        int turn = tiles;
        for (int t = 0; t < nt; ++t) {
            for (int i = 0; i < sm.n_seen[t]; i += kTile, ++turn) {
                if (turn % step != w0) continue;
                const int here = min(sm.n_seen[t] - i, kTile);
                auto from = [&](const uint16_t* p, int r) {
                    return p + base + sm.seen[t][i + min(r, here - 1)] * stride;
                };
                uint4 k[2][D / 32], v[4][D / 64];
                load_keys_bf16<D>(k, [&](int r) { return from(a.tree[0], r); }, g, c, a.wide);
                // The value operand's channels follow the accumulators' order.
                if (FP8) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint16_t* p =
                            from(a.tree[1], 2 * c + (r & 1) + 8 * (r >> 1)) + g * (D / 8);
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) v[r][h] = ptx::ld_stream(p + 8 * h);
                    }
                } else {
                    load_values_bf16<D>(v, [&](int r) { return from(a.tree[1], r); }, g, c);
                }
                float x[NT][4];
                scores_bf16<D, NT>(x, k, sm.q[FP8 ? 1 : 0], g, c);
                bool mine[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[n][j] *= a.scale_log2;
#pragma unroll
                    for (int j = 0; j < 2; ++j) mine[n][j] = (token[n][j] >> t & 1u) != 0;
                }
                hide<NT>(x, here, g);
                hide_others<NT>(x, mine);
                clear_values(v, here, c);
                follow(st, x);
                exponents(st, x);
                if (FP8 && sref == kNoScale) sref = 0;
                add_values_bf16<D, NT>(st, x, v, FP8 ? pow2(kLift - sref) : 1.0f, mine,
                                       nt > 1 && not_finite<false>(v));
            }
        }
    }

    // ---- this warp's rows to shared memory
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
                sm.part_m[warp][r] = st.m[n][i];
                sm.part_l[warp][r] = l;
            }
#pragma unroll
            for (int d = 0; d < D / 16; d += 2) {
                const int ch = FP8 ? channel_fp8<D>(d, g) : channel_bf16<D>(d, g);
                *reinterpret_cast<float4*>(&sm.part[warp][r][ch]) =
                    make_float4(st.o[n][d][i] * unit_of, st.o[n][d][i + 2] * unit_of,
                                st.o[n][d + 1][i] * unit_of, st.o[n][d + 1][i + 2] * unit_of);
            }
        }
    __syncthreads();
    // ---- the CTA's rows, then (S > 1) the cluster's: four channels to a thread
    constexpr int kQuads = D / 4;
    for (int i = tid; i < rows * kQuads; i += kThreads) {
        const int r = i / kQuads, d = i % kQuads * 4;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.part_m[w][r]);
        float l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = sm.part_m[w][r];
            if (mw == -INFINITY) continue;
            const float f = ex2(mw - m);
            l += f * sm.part_l[w][r];
            const float4 y = *reinterpret_cast<const float4*>(&sm.part[w][r][d]);
            o.x += f * y.x;
            o.y += f * y.y;
            o.z += f * y.z;
            o.w += f * y.w;
        }
        *reinterpret_cast<float4*>(&sm.mine[r][d]) = o;
        if (d == 0) {
            sm.mine_m[r] = m;
            sm.mine_l[r] = l;
        }
    }
    if (S > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    for (int i = rank * kThreads + tid; i < rows * kQuads; i += S * kThreads) {
        const int r = i / kQuads, d = i % kQuads * 4;
        const uint32_t at_m = ptx::smem_u32(&sm.mine_m[r]), at_l = ptx::smem_u32(&sm.mine_l[r]);
        const uint32_t at_o = ptx::smem_u32(&sm.mine[r][d]);
        float m = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < S; ++s) m = fmaxf(m, ptx::ld_cluster(ptx::map_rank(at_m, s)));
        for (int s = 0; s < S; ++s) {
            const float ms = ptx::ld_cluster(ptx::map_rank(at_m, s));
            if (ms == -INFINITY) continue;
            const float f = ex2(ms - m);
            l += f * ptx::ld_cluster(ptx::map_rank(at_l, s));
            const float4 y = ptx::ld_cluster_v4(ptx::map_rank(at_o, s));
            o.x += f * y.x;
            o.y += f * y.y;
            o.z += f * y.z;
            o.w += f * y.w;
        }
        const bool none = m == -INFINITY;
        const float inv = none ? 0.0f : 1.0f / l;
        const size_t row = row_of(r);
        *reinterpret_cast<uint2*>(a.out + row * D + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (d == 0) a.lse[row] = none ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
    }
    if (S > 1) ptx::cluster_sync();  // (other CTAs may still read this one's rows)
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

template <int D, bool FP8, int NT>
int launch(const Args& a, long long units, int sms, cudaStream_t stream) {
    using Sh = Shape<NT>;
    const size_t smem = sizeof(Smem<D, NT>) +
                        static_cast<size_t>(a.tokens) * a.n_blocks * sizeof(Entry);
    const auto kernel = blocks_kernel<D, FP8, NT>;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess ||
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return TREE_ATTN_ERR_CUDA;
    // CTAs of a cluster: as many as the SMs hold at once, while each warp has a tile.
    const long long most = a.n_blocks < a.max_pages ? a.n_blocks : a.max_pages;
    const long long tiles = most * (a.P / kTile) + (a.T + kTile - 1) / kTile;
    int S = 1;
    while (S < 16 && 2 * S * units <= static_cast<long long>(Sh::kResident) * sms &&
           tiles >= 2LL * S * Sh::kWarps)
        S *= 2;
    return rc_of(launch_cluster(kernel, dim3(static_cast<unsigned>(units * S)),
                                dim3(Sh::kThreads), smem, S, stream, a));
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
    a.tokens = tokens;
    a.groups = groups;
    a.wide = ptr_aligned(k_pages, 32) && ptr_aligned(tree_k, 32);
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.status = status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f = k_scales != nullptr;
    if (d == 128) {
        if (NT == 1) return f ? launch<128, true, 1>(a, units, sms, s) : launch<128, false, 1>(a, units, sms, s);
        return f ? launch<128, true, 2>(a, units, sms, s) : launch<128, false, 2>(a, units, sms, s);
    }
    if (NT == 1) return f ? launch<64, true, 1>(a, units, sms, s) : launch<64, false, 1>(a, units, sms, s);
    return f ? launch<64, true, 2>(a, units, sms, s) : launch<64, false, 2>(a, units, sms, s);
}
