// verify_fp8.cu -- split tree attention over the 8-bit paged cache: a prefix pass
// over the committed rows, which leaves partial results, then a kernel that
// attends the tree tokens and merges everything by log-sum-exp.
//
// Prefix pass.  For a unit (sequence, KV head) with R query rows (tree nodes x grouped heads)
// and keys j held as codes with scales:
//   x_rj = c_r F_j <2^u_r q_r, k_j>,  F_j = 2^(scale of k_j),
//   c_r = softmax scale log2(e) 2^-u_r
//   out_r = sum_j 2^x_rj v_j / sum_j 2^x_rj.
// Both products are turned round:
//   S^T = K Q^T     (128 keys x rows; A = K tile, B = Q)
//   O^T += V^T P^T  (d x rows;        A = V tile, B = P)
// * The key codes go to the tensor cores as they are, so the queries have to be
//   8 bits as well: a query row enters as two e4m3 rows, the rounded value (hi)
//   and what is left of it (lo), summed in one accumulator.  Each row has a power of
//   two 2^u of its own, so that a large query costs the other rows nothing.
// * A probability may be any fraction of its row's largest, and thousands of
//   small ones may make up half of the row (8-bit halves, with a step of 2^-13 of
//   the reference, lost up to 30 % of such a result).  So P is fp16, and warps of
//   their own widen a block's value codes to fp16, which is exact.
// * A TMEM lane is a key, so a key's scales are scalars of the thread that
//   holds it, and the softmax has no idle lanes however few rows there are.
// * The value scale joins the exponent: e = x + scale of v_j, p = 2^(e - ref),
//   O sums p v, and the row's sum takes p 2^-(scale of v_j) in fp32.
// * A row's maximum would need the 128 lanes to meet; instead each block only
//   asks whether any e exceeds its row's reference by more than 15 (p must stay
//   below 2^16): each warpgroup asks for its own rows.  If one does, its references
//   move and O is rescaled (the first block of a segment always does that).
// * A new reference leaves the largest p at 2^7.  fp16 rounds to 11 bits down to
//   2^-14 and to half of 2^-24 below, and a code is at most 448, so with n keys the
//   result is off by
//     2^-11 sum_j p_j |v_j| / l + n 2^-31 max_j (p_j max|v_j|) / l
//   at most: the second term, of keys whose p leaves fp16's normal range, is 2^-17
//   of max|v| for 16384 keys and 2^-11 for a million.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/tree_attn.h"
#include "fp8.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "layout.h"
#include "ptx_serving.cuh"
#include "tma_host.h"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kKeys = 2 * kChunk;  // keys of a block
// p = 2^(e - reference) may reach 2^kMost.  When a block passes that, the references
// of all rows whose largest p stands above 2^kFresh move up until it is that, so that
// rows close to their limit do not stop a later block.  kFresh 5 would leave fewer
// blocks to be done twice (4 x 32768 tokens, 80 rows: 86 us for 89), but four times
// the fixed error of small p.
constexpr float kMost = 15.f, kFresh = 7.f;
// Work-line slots (64-token steps) that stand for a segment's fixed cost.  Measured, 64
// sequences of up to 16384 tokens, 4 rows a head: 4: 185 us, 6: 178.5, 8: 178.8, 12: 181;
// 4 x 32768 tokens, 80 rows: 90.5, 89.3, 89.0, 89.4 us.
constexpr int kOverhead = 8;

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

struct Fp8Args {
    const uint16_t* q;
    const uint8_t* k_scales;
    const uint8_t* v_scales;
    const int32_t* block_table;
    const int32_t* seq_lens;
    float* ws;
    int32_t* status;
    int B, Hq, Hkv, G, T, M, RB, P, max_pages, num_pages, n_ctas, ovh;
    float scale_log2;
    unsigned long long wait_ns;
};

// Shared memory and TMEM of a CTA for D-wide heads and tiles of up to R rows,
// split over WG softmax warpgroups.
template <int D, int R, int WG>
struct Shape {
    static constexpr int H = R / WG;                  // rows of a warpgroup
    static constexpr int WARPS = 4 * WG;              // softmax warps
    // And the warps for copies, MMAs and values; with many rows to a thread these
    // make one warpgroup, which gives its registers to the softmax.
    static constexpr bool SHIFT = H > 32;
    // Warps that widen values (64 sequences of up to 16384 tokens, 16 rows: 2: 176 us,
    // 4: 179, 8: 183; one of 8192 tokens, 48 rows: 17.6, 18.1, 18.3).
    static constexpr int WIDEN = 2;
    static constexpr int THREADS = 32 * (WARPS + 2 + WIDEN);
    // (8 x 16384 tokens, 80 rows: 184 registers 97.8 us, 200: 98.1, 208: 98.9; 128 rows:
    // 145, 145, 137.)
    static constexpr int SOFT_REGS = H > 48 ? 208 : 184, HELP_REGS = H > 48 ? 88 : 136;
    static_assert(!SHIFT || (WG == 2 && 256 * SOFT_REGS + 128 * HELP_REGS <= 384 * 168),
                  "registers at launch");
    static constexpr int TILE = kKeys * D;            // K (or V) codes of a block
    static constexpr int STAGE = 2 * TILE;
    static constexpr int Q_BYTES = 2 * R * D;         // both halves of each row
    static constexpr int PB = 2 * R;                  // bytes of a key's row of P
    static constexpr int PW = PB <= 32 ? 32 : (PB <= 64 ? 64 : 128);  // row bytes of a P tile
    static constexpr int P_ATOM = kKeys * PW;
    static constexpr int P_BYTES = (PB > 128 ? 2 : 1) * P_ATOM;
    static constexpr int V_ATOM = kKeys * 128;        // 64 columns of the fp16 values
    static constexpr int V_BYTES = D / 64 * V_ATOM;
    // Buffers of fp16 values: with many rows at d = 128 there is room for one, filled
    // between the P.V products of two blocks.
    static constexpr int NV = D == 128 && R > 64 ? 1 : 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + (Q_BYTES + 1023) / 1024 * 1024;
    static constexpr int OFF_V = OFF_P + 2 * P_BYTES;
    static constexpr int OFF_STAGE = OFF_V + NV * V_BYTES;
    static constexpr int SMALL = 8 * 1024;            // scales, references, barriers
    static constexpr int FIT = (227 * 1024 - 1024 - SMALL - OFF_STAGE) / STAGE;
    static constexpr int MOST = D == 128 ? 6 : 8;
    static constexpr int NS = FIT > MOST ? MOST : FIT;  // ring depth
    static constexpr int OFF_SCALE = OFF_STAGE + NS * STAGE;  // [NS][K, V][128]
    static constexpr int OFF_REF = OFF_SCALE + NS * 2 * kKeys;  // reference, factor of each row
    static constexpr int OFF_ALPHA = OFF_REF + R * 8;           // its last change, as a factor
    static constexpr int OFF_WMAX = OFF_ALPHA + R * 4;          // [4][R]: maxima / sums by warp
    static constexpr int OFF_MISC = OFF_WMAX + 4 * R * 4;
    static constexpr int OFF_BAR = OFF_MISC + 192;
    // barriers
    static constexpr int KV_FULL = 0;
    static constexpr int KV_EMPTY = NS;
    static constexpr int S_FULL = 2 * NS;
    static constexpr int S_FREE = S_FULL + 2;
    static constexpr int P_FULL = S_FULL + 4;
    static constexpr int P_FREE = S_FULL + 6;
    static constexpr int O_FULL = S_FULL + 8;
    static constexpr int O_FREE = S_FULL + 9;
    static constexpr int Q_FULL = S_FULL + 10;
    static constexpr int MEET = S_FULL + 11;   // the softmax warps meet
    static constexpr int SEG_FULL = S_FULL + 12;   // [2]: a segment has been announced
    static constexpr int SEG_EMPTY = S_FULL + 14;  // [2]: every reader has it
    static constexpr int DRAIN = S_FULL + 16;
    static constexpr int CHECK = S_FULL + 17;       // [WG]: a warpgroup's vote on a block
    static constexpr int MEET_WG = CHECK + WG;      // [WG]: a warpgroup meets
    static constexpr int V_FULL = MEET_WG + WG;     // [NV]: a block's values are fp16
    static constexpr int NBAR = V_FULL + NV;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 1024;  // + alignment slack
    // TMEM columns: S in two buffers, then O.
    static constexpr int NB = 2;
    static constexpr int TM_S = 0;
    static constexpr int TM_O = NB * R;
    static_assert(R % WG == 0 && H % 8 == 0 && R <= kRows, "rows of a tile");
    static_assert(NB * R + R <= 512, "TMEM budget");
    static_assert(NS >= 2 && SMEM <= 227 * 1024, "shared memory budget");
    static_assert(SMEM > 114 * 1024, "one CTA per SM keeps TMEM allocation uncontended");
    static_assert(OFF_BAR + NBAR * 8 - OFF_SCALE <= SMALL, "small arrays fit their room");
};

// A piece of a unit's keys that this CTA takes, as the copies' warp announces it.
struct Piece {
    int b, hk, rb, slot;         // slot of its partial; -1: no more pieces
    int chunk_begin, chunk_end;  // 64-token steps of the sequence
    int L, pad;                  // committed tokens
};

struct Misc {
    uint32_t tmem_base;
    int abort;
    int pad[2];
    Piece piece[2];
    uint8_t vote[2][32];  // by warp: a probability left its range
};
static_assert(sizeof(Misc) <= 192, "Misc fits its slot");

// tcgen05 instruction descriptor for fp32 D and A and B of format 0: e4m3 in
// kind::f8f6f4, fp16 in kind::f16.
TA_HD uint32_t idesc_0_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
           ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// Shared-memory descriptor of a tile whose rows are W = 128, 64 or 32 bytes, with
// the swizzle of that width (modes 2, 4, 6).  8-row groups are 8 * W bytes apart
// (the stride dimension for K-major and MN-major alike: a row holds W bytes of K,
// or of M/N); `lbo`: bytes between W-byte columns of an MN-major tile.
template <int W>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lbo = 16) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) |
           (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>((8 * W) >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(W == 128 ? 2 : (W == 64 ? 4 : 6)) << 61);
}

// Byte offset of 16-byte chunk c of row r in such a tile.
template <int W>
__device__ __forceinline__ uint32_t tile_offset(uint32_t r, uint32_t c) {
    const uint32_t x = W == 128 ? (r & 7u) : (W == 64 ? ((r >> 1) & 3u) : ((r >> 2) & 1u));
    return r * W + ((c ^ x) << 4);
}

struct Range {
    long long x0, x1, base0;
    int b0;
    int32_t lraw0;
};

// This CTA's stretch of the work line (one warp; every lane gets it).
__device__ Range plan_range(const Fp8Args& a, int lane) {
    const int upb = a.Hkv * a.RB;
    auto len_of = [&](int b) -> int {
        if (b >= a.B) return 0;
        bool bad;
        const int n = unit_len(unit_chunks(a.seq_lens[b], a.P, a.max_pages, kTreeNone, 0, bad),
                               a.ovh);
        if (bad && blockIdx.x == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
        return n;
    };
    const int n0 = len_of(lane), n1 = len_of(lane + 32);  // both loads in flight
    long long tot = __reduce_add_sync(kFull, n0) + __reduce_add_sync(kFull, n1);
    for (int b = 64; b < a.B; b += 32) tot += __reduce_add_sync(kFull, len_of(b + lane));
    const long long W = tot * upb;
    Range r;
    r.x0 = cta_start(blockIdx.x, W, a.n_ctas);
    r.x1 = cta_start(blockIdx.x + 1, W, a.n_ctas);
    r.b0 = 0;
    r.base0 = 0;
    r.lraw0 = 0;
    if (r.x0 >= r.x1) return r;
    long long run = 0;
    for (int b = 0; b < a.B; b += 32) {
        const long long n =
            static_cast<long long>(upb) * (b == 0 ? n0 : (b == 32 ? n1 : len_of(b + lane)));
        long long incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(kFull, incl, off);
            if (lane >= off) incl += v;
        }
        const bool hit = run + incl - n <= r.x0 && r.x0 < run + incl;
        const unsigned m = __ballot_sync(kFull, hit);
        if (m != 0) {
            const int src = __ffs(m) - 1;
            r.b0 = b + src;
            r.base0 = run + __shfl_sync(kFull, incl - n, src);
            r.lraw0 = a.seq_lens[r.b0];
            break;
        }
        run += __shfl_sync(kFull, incl, 31);
    }
    return r;
}

// Reduces NC columns, held one value per lane and column, over the 32 lanes
// (op: of two values).  Afterwards v[i] of lane l is that of column 32 i + l, for
// columns below NC.  Each exchange halves the columns a lane still holds.
template <int NC, typename Op>
__device__ __forceinline__ void reduce_columns(float* v, int lane, Op op) {
    if constexpr (NC > 32) {
        reduce_columns<32>(v, lane, op);
        reduce_columns<NC - 32>(v + 32, lane, op);
        v[1] = v[32];
    } else if constexpr (NC == 24) {
        reduce_columns<16>(v, lane, op);
        reduce_columns<8>(v + 16, lane, op);
        if (lane >= 16) v[0] = v[16];
    } else {
        static_assert(NC == 8 || NC == 16 || NC == 32, "columns");
#pragma unroll
        for (int w = NC / 2; w >= 1; w >>= 1) {
            const bool up = (lane & w) != 0;
#pragma unroll
            for (int i = 0; i < w; ++i) {
                const float send = up ? v[i] : v[i + w];
                const float keep = up ? v[i + w] : v[i];
                v[i] = op(keep, __shfl_xor_sync(kFull, send, w));
            }
        }
#pragma unroll
        for (int w = NC; w < 32; w <<= 1) v[0] = op(v[0], __shfl_xor_sync(kFull, v[0], w));
    }
}

// The scores of one key and H rows.
template <int H>
__device__ __forceinline__ void load_scores(uint32_t ta, float* x) {
    static_assert(H % 8 == 0, "columns");
#pragma unroll
    for (int c = 0; c < H / 32; ++c) ptx::tmem_ld32(ta + 32 * c, x + 32 * c);
    constexpr int c16 = H / 32 * 32;
    if constexpr (H % 32 >= 16) ptx::tmem_ld16(ta + c16, x + c16);
    constexpr int c8 = H / 16 * 16;
    if constexpr (H % 16 == 8) ptx::tmem_ld8(ta + c8, x + c8);
    ptx::tmem_wait_ld();
}

__device__ __forceinline__ int blocks_of(const Piece& sg) {
    return (sg.chunk_end - sg.chunk_begin + 1) / 2;
}

template <int D, int R, int WG>
__global__ void __launch_bounds__((Shape<D, R, WG>::THREADS), 1)
    prefix_fp8_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Fp8Args a) {
    using S = Shape<D, R, WG>;
    constexpr int kWarpTma = S::WARPS, kWarpMma = S::WARPS + 1;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sb = raw_addr + pad;
    Misc* misc = reinterpret_cast<Misc*>(smem + S::OFF_MISC);
    volatile int* abort_flag = &misc->abort;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sb + S::OFF_BAR + 8u * i; };

    if (warp == kWarpTma && lane == 0) {
        for (int s = 0; s < S::NS; ++s) {
            ptx::mbar_init(bar(S::KV_FULL + s), 1);
            ptx::mbar_init(bar(S::KV_EMPTY + s), S::WARPS + S::WIDEN);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(S::S_FULL + i), 1);
            ptx::mbar_init(bar(S::S_FREE + i), S::WARPS);
            ptx::mbar_init(bar(S::P_FULL + i), S::WARPS);
            ptx::mbar_init(bar(S::P_FREE + i), 1);
        }
        ptx::mbar_init(bar(S::O_FULL), 1);
        ptx::mbar_init(bar(S::O_FREE), S::WARPS);
        ptx::mbar_init(bar(S::Q_FULL), S::WARPS);
        for (int i = 0; i < WG; ++i) {
            ptx::mbar_init(bar(S::CHECK + i), 4);
            ptx::mbar_init(bar(S::MEET_WG + i), 4);
        }
        ptx::mbar_init(bar(S::MEET), S::WARPS);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(S::SEG_FULL + i), 1);
            ptx::mbar_init(bar(S::SEG_EMPTY + i), S::WARPS + 1 + S::WIDEN);
        }
        for (int i = 0; i < S::NV; ++i) ptx::mbar_init(bar(S::V_FULL + i), S::WIDEN);
        ptx::mbar_init(bar(S::DRAIN), 1);
        misc->abort = 0;
        for (int i = 0; i < 16; ++i) reinterpret_cast<uint32_t*>(misc->vote)[i] = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(ptx::smem_u32(&misc->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    const uint64_t pol = ptx::policy_evict_first();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc->tmem_base;
    // Everything below reads inputs that the kernel before may write.  Only
    // after that wait may the next kernel start (see tree_mask_kernel).
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    auto fail = [&]() {
        *abort_flag = 1;
        report(a.status, TREE_ATTN_STATUS_TIMEOUT);
    };

    // Announced piece number k, for all warps but the copies'; false: no more, or a
    // wait ran out.
    auto next_piece = [&](uint32_t k, Piece& pc) -> bool {
        if (!__all_sync(kFull, ptx::mbar_wait(bar(S::SEG_FULL + (k & 1)), (k >> 1) & 1,
                                              a.wait_ns))) {
            fail();
            return false;
        }
        pc = misc->piece[k & 1];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(S::SEG_EMPTY + (k & 1)));
        return pc.slot >= 0;
    };

    auto copies = [&]() {
        // ================= this CTA's pieces and their copies: lane k < 8 takes
        // box k of a block
        const Range rg = plan_range(a, lane);
        Walker w;
        w.init_known(a.seq_lens, a.B, a.P, a.max_pages, a.Hkv * a.RB, a.RB, rg.b0, rg.base0, rg.x0,
                     rg.x1, kTreeNone, 0, a.ovh, rg.lraw0);
        const int Pb = a.P < kChunk ? a.P : kChunk;  // tokens per box
        const int nsub = kChunk / Pb;                // boxes per 64-token step
        const int pshift = __ffs(a.P) - 1;
        const int hh = (lane >> 2) & 1, sub = lane & 3;
        uint32_t jj = 0;
        bool ok = true;
        Segment sg = {};
#pragma unroll 1
        for (uint32_t k = 0; ok; ++k) {
            const bool more = w.next(sg);
            bool bad;
            const int L = clamp_seq_len(sg.len_raw, a.P, a.max_pages, bad);
            if (k >= 2 && !__all_sync(kFull, ptx::mbar_wait(bar(S::SEG_EMPTY + (k & 1)),
                                                            ((k >> 1) - 1) & 1, a.wait_ns))) {
                fail();
                ok = false;
                break;
            }
            if (lane == 0) {
                Piece pc;
                pc.b = sg.b;
                pc.hk = sg.hk;
                pc.rb = sg.rb;
                pc.slot = more ? sg.unit + static_cast<int>(blockIdx.x) : -1;
                pc.chunk_begin = sg.chunk_begin;
                pc.chunk_end = sg.chunk_end;
                pc.L = L;
                pc.pad = 0;
                misc->piece[k & 1] = pc;
                ptx::mbar_arrive(bar(S::SEG_FULL + (k & 1)));
            }
            __syncwarp();
            if (!more) break;
            const int npages = (L + a.P - 1) >> pshift;
            const int32_t* table = a.block_table + static_cast<size_t>(sg.b) * a.max_pages;
            // 64 table entries from `base` on, two to a lane: looked up long
            // before the block that uses them.
            int base = (sg.chunk_begin * kChunk) >> pshift;
            auto look = [&](int i) -> int { return i < npages ? table[i] : -1; };
            int near_ = look(base + lane), far_ = look(base + 32 + lane);
#pragma unroll 1
            for (int ch = sg.chunk_begin; ch < sg.chunk_end; ch += 2, ++jj) {
                if (((ch * kChunk) >> pshift) - base >= 32) {
                    base += 32;
                    near_ = far_;
                    far_ = look(base + 32 + lane);
                }
                const int tok = (ch + hh) * kChunk + sub * Pb;
                const int lp = tok >> pshift;
                const int at = lp - base;
                const int p0 = __shfl_sync(kFull, near_, at & 31);
                const int p1 = __shfl_sync(kFull, far_, at & 31);
                const int pid = at < 32 ? p0 : p1;
                bool use = lane < 8 && ch + hh < sg.chunk_end && sub < nsub && lp < npages;
                if (use && (pid < 0 || pid >= a.num_pages)) {
                    report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                    use = false;
                }
                const int n = __popc(__ballot_sync(kFull, use));
                const int s = jj % S::NS;
                if (jj >= S::NS &&
                    !__all_sync(kFull, ptx::mbar_wait(bar(S::KV_EMPTY + s), ((jj / S::NS) - 1) & 1,
                                                      a.wait_ns))) {
                    fail();
                    ok = false;
                    break;
                }
                if (__any_sync(kFull, *abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = bar(S::KV_FULL + s);
                if (lane == 0) {
                    if (n > 0)
                        ptx::mbar_arrive_expect_tx(fb, static_cast<uint32_t>(n * Pb * 2 * (D + 1)));
                    else
                        ptx::mbar_arrive(fb);
                }
                __syncwarp();
                if (use) {
                    const uint32_t kst = sb + S::OFF_STAGE + s * S::STAGE;
                    const uint32_t sst = sb + S::OFF_SCALE + s * 2 * kKeys;
                    const int y = (pid * a.Hkv + sg.hk) * a.P + (tok & (a.P - 1));
                    const int row = hh * kChunk + sub * Pb;
                    ptx::tma_load_2d(kst + row * D, &tm_k, 0, y, fb, pol);
                    ptx::bulk_load(sst + row, a.k_scales + y, Pb, fb);
                    ptx::bulk_load(sst + kKeys + row, a.v_scales + y, Pb, fb);
                    ptx::tma_load_2d(kst + S::TILE + row * D, &tm_v, 0, y, fb, pol);
                }
                __syncwarp();
            }
        }
        // Every copy lands before the CTA exits, whoever has given up.
        const uint32_t first = jj > S::NS ? jj - S::NS : 0;
        for (uint32_t j = first; j < jj; ++j)
            (void)ptx::mbar_wait(bar(S::KV_FULL + j % S::NS), (j / S::NS) & 1, ptx::kDrainLimitNs);
    };
    auto products = [&]() {
        // ================= MMA issuer: the whole warp walks, one lane issues.
        // It polls without waiting: a suspended poll for P would hold up the
        // scores of the next block.
        const bool lead = ptx::elect_one();
        const uint32_t id_s = idesc_0_f32(kKeys, R, false, false);
        const uint32_t id_o = idesc_0_f32(D, R, true, true);
        uint32_t jj = 0, kk = 0;
        bool ok = true;
        Piece sg;
        while (ok && next_piece(kk, sg)) {
            if (!__all_sync(kFull, ptx::mbar_wait(bar(S::Q_FULL), kk & 1, a.wait_ns))) {
                fail();
                break;
            }
            ptx::tc_fence_after();
            const int n = blocks_of(sg);
            int nq = 0, np = 0;
            uint64_t t0 = 0;
            while (np < n) {
                bool progress = false;
                if (np < nq) {
                    const uint32_t j = jj + np;
                    const bool go =
                        ptx::mbar_test(bar(S::P_FULL + (j & 1)), (j >> 1) & 1) &&
                        ptx::mbar_test(bar(S::V_FULL + j % S::NV), (j / S::NV) & 1) &&
                        (np > 0 || kk == 0 || ptx::mbar_test(bar(S::O_FREE), (kk - 1) & 1));
                    if (__all_sync(kFull, go)) {
                        ptx::tc_fence_after();
                        const uint32_t vst = sb + S::OFF_V + (j % S::NV) * S::V_BYTES;
                        const uint32_t pst = sb + S::OFF_P + (j & 1) * S::P_BYTES;
                        // A block of one 64-token step has nothing in its second half.
                        const int nk = sg.chunk_end - sg.chunk_begin - 2 * np >= 2 ? 8 : 4;
                        if (lead) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                if (k >= nk) break;
                                ptx::mma_f16(tmem + S::TM_O,
                                             tile_desc<128>(vst + k * 16 * 128, S::V_ATOM),
                                             tile_desc<S::PW>(pst + k * 16 * S::PW, S::P_ATOM),
                                             id_o, (np == 0 && k == 0) ? 0u : 1u);
                            }
                            ptx::mma_commit(bar(S::P_FREE + (j & 1)));
                        }
                        __syncwarp();
                        ++np;
                        progress = true;
                    }
                }
                if (nq < n) {
                    const uint32_t j = jj + nq;
                    const int s = j % S::NS;
                    const int sbuf = j % S::NB;
                    const bool go =
                        ptx::mbar_test(bar(S::KV_FULL + s), (j / S::NS) & 1) &&
                        (j < S::NB ||
                         ptx::mbar_test(bar(S::S_FREE + sbuf), ((j / S::NB) - 1) & 1));
                    if (__all_sync(kFull, go)) {
                        ptx::tc_fence_after();
                        const uint32_t kst = sb + S::OFF_STAGE + s * S::STAGE;
                        if (lead) {
#pragma unroll
                            for (int k = 0; k < 2 * D / 32; ++k) {
                                const int kd = k % (D / 32);  // the hi rows, then the lo rows
                                ptx::mma_f8(tmem + S::TM_S + sbuf * R, tile_desc<D>(kst + kd * 32),
                                            tile_desc<D>(sb + S::OFF_Q + (k / (D / 32)) * R * D +
                                                         kd * 32),
                                            id_s, k > 0 ? 1u : 0u);
                            }
                            ptx::mma_commit(bar(S::S_FULL + sbuf));
                        }
                        __syncwarp();
                        ++nq;
                        progress = true;
                    }
                }
                if (progress) {
                    t0 = 0;
                } else {
                    const uint64_t now = ptx::globaltimer();
                    if (t0 == 0) t0 = now;
                    if (__any_sync(kFull, now - t0 > a.wait_ns || *abort_flag)) {
                        ok = false;
                        break;
                    }
                }
            }
            if (!ok) {
                fail();
                break;
            }
            if (lead) ptx::mma_commit(bar(S::O_FULL));
            __syncwarp();
            jj += n;
            ++kk;
        }
        if (lead) ptx::mma_commit(bar(S::DRAIN));
        __syncwarp();
        (void)ptx::mbar_wait(bar(S::DRAIN), 0, ptx::kDrainLimitNs);
    };
    auto values = [&]() {
        // ================= values: a lane widens the codes of a key to fp16.
        // A key past the data gets zeros, as 0 * NaN is not 0.
        uint32_t jj = 0, kk = 0;
        uint32_t stage = 0, phase = 0;  // jj % NS, (jj / NS) & 1
        bool ok = true;
        Piece sg;
        while (ok && next_piece(kk, sg)) {
#pragma unroll 1
            for (int ch = sg.chunk_begin; ch < sg.chunk_end; ch += 2, ++jj) {
                const int rows = min(2, sg.chunk_end - ch) * kChunk;
                const int keys = min(rows, sg.L - ch * kChunk);
                // The codes have landed; P.V of the block before in this buffer has
                // completed.
                bool in = ptx::mbar_wait(bar(S::KV_FULL + stage), phase, a.wait_ns);
                if (jj >= S::NV)
                    in &= ptx::mbar_wait(bar(S::P_FREE + ((jj - S::NV) & 1)),
                                         ((jj - S::NV) >> 1) & 1, a.wait_ns);
                if (!__all_sync(kFull, in)) {
                    fail();
                    ok = false;
                    break;
                }
                const uint32_t src = sb + S::OFF_STAGE + stage * S::STAGE + S::TILE;
                const uint32_t dst = sb + S::OFF_V + (jj % S::NV) * S::V_BYTES;
#pragma unroll 1
                for (int key = (warp - kWarpMma - 1) * 32 + lane; key < rows;
                     key += S::WIDEN * 32) {
                    uint4 v[D / 16];
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        v[c] = ptx::ld_shared_v4(src + tile_offset<D>(key, c));
                        if (key >= keys) v[c] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t w[8];
                        f16x2_of_e4m3x4(v[c].x, w[0], w[1]);
                        f16x2_of_e4m3x4(v[c].y, w[2], w[3]);
                        f16x2_of_e4m3x4(v[c].z, w[4], w[5]);
                        f16x2_of_e4m3x4(v[c].w, w[6], w[7]);
                        const uint32_t at = dst + (c >> 2) * S::V_ATOM;
                        ptx::st_shared_v4(at + tile_offset<128>(key, (2 * c) & 7), w[0], w[1],
                                          w[2], w[3]);
                        ptx::st_shared_v4(at + tile_offset<128>(key, (2 * c + 1) & 7), w[4], w[5],
                                          w[6], w[7]);
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(bar(S::V_FULL + jj % S::NV));
                    ptx::mbar_arrive(bar(S::KV_EMPTY + stage));
                }
                if (++stage == S::NS) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            ++kk;
        }
    };
    if (warp >= S::WARPS) {
        if constexpr (S::SHIFT)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::HELP_REGS));
        if (warp == kWarpTma)
            copies();
        else if (warp == kWarpMma)
            products();
        else
            values();
    } else {
        // ================= softmax and epilogue
        if constexpr (S::SHIFT)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::SOFT_REGS));
        constexpr int H = S::H;     // this warpgroup's rows
        const int wg = warp >> 2;
        const int quad = warp & 3;  // the TMEM lanes this warp reaches
        const int key = quad * 32 + lane;
        const int row0 = wg * H;    // first row of the tile taken here
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        // By pairs of rows: minus their references, then their factors c_r.
        float4* row_pair = reinterpret_cast<float4*>(smem + S::OFF_REF);
        auto nref = [&](int r) -> float& {
            return reinterpret_cast<float*>(row_pair)[(r >> 1) * 4 + (r & 1)];
        };
        auto factor = [&](int r) -> float& {
            return reinterpret_cast<float*>(row_pair)[(r >> 1) * 4 + 2 + (r & 1)];
        };
        float* alpha = reinterpret_cast<float*>(smem + S::OFF_ALPHA);
        float* wmax = reinterpret_cast<float*>(smem + S::OFF_WMAX);  // [4][R]
        auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
            // A role that gave up leaves its barriers unfinished, so those who
            // wait for it give up within the limit too.
            const bool all = __all_sync(kFull, ptx::mbar_wait(b, parity, a.wait_ns));
            if (!all) fail();
            return all;
        };
        uint32_t met = 0;  // meetings of the softmax warps so far
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(S::MEET));
            const uint32_t parity = met & 1;
            ++met;
            return wait_all(bar(S::MEET), parity);
        };

        uint32_t met_wg = 0;
        auto meet_wg = [&]() -> bool {  // the same of a warpgroup, whose rows are its own
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(S::MEET_WG + wg));
            const uint32_t parity = met_wg & 1;
            ++met_wg;
            return wait_all(bar(S::MEET_WG + wg), parity);
        };

        uint32_t jj = 0, kk = 0;
        uint32_t stage = 0, phase = 0;  // jj % NS, (jj / NS) & 1
        bool ok = true;
        Piece cur;
        while (ok && next_piece(kk, cur)) {
            const int L = cur.L;
            const int Mrb = min(kRows, a.M - cur.rb * kRows);  // query rows of the tile
            // ---- the tile's queries: a row's power of two brings its largest |q| into
            // (224, 448]; each value is held as hi + lo, exactly down to 2^-2 and to
            // 2^-10 below (2^-17 of the row's largest at the most).
            {
                constexpr int LPR = D / 8;                   // lanes per row
                constexpr int STEP = S::WARPS * 32 / LPR;    // rows per pass
                constexpr int NP = (R + STEP - 1) / STEP;
                const int r0 = threadIdx.x / LPR, gl = threadIdx.x % LPR;
                uint4 x[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    // (loads that no branch surrounds are all in flight at once)
                    const int r = r0 + i * STEP;
                    const int rr = cur.rb * kRows + min(r, Mrb - 1);
                    const int t = rr / a.G, h = cur.hk * a.G + rr % a.G;
                    x[i] = __ldg(reinterpret_cast<const uint4*>(
                        a.q + ((static_cast<size_t>(cur.b) * a.T + t) * a.Hq + h) * D + gl * 8));
                }
                uint8_t* qs = smem + S::OFF_Q;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int r = r0 + i * STEP;
                    if (r >= Mrb) x[i] = make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t wd[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t m = 0;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t lo = (wd[u] << 16) & 0x7fff0000u, hi = wd[u] & 0x7fff0000u;
                        if (lo < 0x7f800000u) m = max(m, lo);
                        if (hi < 0x7f800000u) m = max(m, hi);
                    }
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1)
                        m = max(m, __shfl_xor_sync(kFull, m, off));
                    if (r >= R) continue;
                    int kq = m == 0 ? 0
                                    : 134 - static_cast<int>(m >> 23) +
                                          ((m & 0x7fffffu) <= 0x600000u ? 1 : 0);
                    kq = kq > 100 ? 100 : kq;
                    const float up = __int_as_float((127 + kq) << 23);
                    if (gl == 0) factor(r) = a.scale_log2 * __int_as_float((127 - kq) << 23);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float v0 = __uint_as_float(wd[u] << 16) * up;
                        float v1 = __uint_as_float(wd[u] & 0xffff0000u) * up;
                        // an infinite query has no finite scores: NaN, as its softmax
                        v0 = fabsf(v0) < 1e30f ? v0 : __int_as_float(0x7fffffff);
                        v1 = fabsf(v1) < 1e30f ? v1 : __int_as_float(0x7fffffff);
                        hi[u] = e4m3x2(v0, v1);
                        const uint32_t hh = f16x2_of_e4m3x2(hi[u]);
                        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hh));
                        lo[u] = e4m3x2(v0 - b.x, v1 - b.y);
                    }
                    // tile rows: all hi halves, then all lo halves
                    uint8_t* at = qs + tile_offset<D>(r, gl >> 1) + (gl & 1) * 8;
                    *reinterpret_cast<uint2*>(at) =
                        make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                    *reinterpret_cast<uint2*>(at + R * D) =
                        make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(S::Q_FULL));
                if (!meet()) {  // the factors, beside the first score product
                    ok = false;
                    break;
                }
            }

            float l[H];  // the rows' sums over this thread's keys
#pragma unroll
            for (int i = 0; i < H; ++i) l[i] = 0.f;
            float x[H];  // scores of this thread's key, then its probabilities
            // Moves the references up to 2^kFresh below block q's largest e where that
            // stands above (all rows' in a first block), and rescales l and O.
            auto move_refs = [&](uint32_t q, bool first, bool valid, float F, float vs) -> bool {
                load_scores<H>(lanes + S::TM_S + (q & 1) * R + row0, x);
                // largest e of every row, by warp, then by warpgroup (fmaxf passes over NaN)
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const float4 rp = row_pair[(row0 + i) >> 1];
                    x[i] = valid ? fmaf(x[i] * F, rp.z, vs) : kNegInf;
                    x[i + 1] = valid ? fmaf(x[i + 1] * F, rp.w, vs) : kNegInf;
                }
                reduce_columns<H>(x, lane, [](float u, float v) { return fmaxf(u, v); });
#pragma unroll
                for (int i = 0; i < (H + 31) / 32; ++i)
                    if (i * 32 + lane < H) wmax[quad * R + row0 + i * 32 + lane] = x[i];
                if (!meet_wg()) return false;
                const int r = row0 + (threadIdx.x & 127);
                if (r < row0 + H) {
                    const float top = fmaxf(fmaxf(wmax[r], wmax[R + r]),
                                            fmaxf(wmax[2 * R + r], wmax[3 * R + r])) -
                                      kFresh;
                    // (a first block of NaN scores has no largest: any finite reference)
                    const float old = first ? kNegInf : -nref(r);
                    const float now = top > old ? top : (first ? 0.f : old);
                    nref(r) = -now;
                    alpha[r] = ptx::ex2(old - now);
                }
                if (!meet_wg()) return false;
                if (first) return true;
                // O holds the blocks before once P.V of the last has completed.
                if (!wait_all(bar(S::P_FREE + ((q - 1) & 1)), ((q - 1) >> 1) & 1)) return false;
                ptx::tc_fence_after();
#pragma unroll
                for (int c = 0; c < H; c += 8) {
                    float al[8];
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        al[i] = alpha[row0 + c + i];
                        any |= al[i] != 1.f;
                    }
                    if (!any) continue;  // the same for the whole warpgroup
                    const uint32_t to = lanes + S::TM_O + row0 + c;
                    float o[8];
                    ptx::tmem_ld8(to, o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        l[c + i] *= al[i];
                        o[i] *= al[i];
                    }
                    ptx::tmem_st8(to, o);
                }
                ptx::tmem_wait_st();
                return true;
            };
            // Block q's probabilities p = 2^(c F s + vs - reference), into x and, as fp16,
            // into the key's row of the P tile; a key past the data has none.  Returns
            // whether a p has passed 2^kMost (NaN has not).
            auto probabilities = [&](uint32_t q, bool valid, float F, float vs) -> bool {
                const uint64_t F2 = ptx::f2_pack(F, F), vs2 = ptx::f2_pack(vs, vs);
                const uint32_t prow = sb + S::OFF_P + (q & 1) * S::P_BYTES;
                // 16-byte chunk of the key's row for rows i .. i + 7
                auto p_at = [&](int i) -> uint32_t {
                    const int c = wg * (H / 8) + i / 8;
                    return prow + (c * 16 / S::PW) * S::P_ATOM +
                           tile_offset<S::PW>(key, c % (S::PW / 16));
                };
                load_scores<H>(lanes + S::TM_S + (q & 1) * R + row0, x);
                __half2 top = __float2half2_rn(0.f);
#pragma unroll
                for (int i = 0; i < H; i += 8) {
                    uint32_t ph[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int k = i + 2 * u;
                        const float4 rp = row_pair[(row0 + k) >> 1];
                        float e0, e1;
                        ptx::f2_unpack(ptx::f2_fma(ptx::f2_mul(ptx::f2_pack(x[k], x[k + 1]), F2),
                                                   ptx::f2_pack(rp.z, rp.w),
                                                   ptx::f2_add(vs2, ptx::f2_pack(rp.x, rp.y))),
                                       e0, e1);
                        x[k] = ptx::ex2(e0);
                        x[k + 1] = ptx::ex2(e1);
                        const __half2 h = __floats2half2_rn(x[k], x[k + 1]);
                        top = __hmax2(top, h);
                        ph[u] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    ptx::st_shared_v4(p_at(i), ph[0], ph[1], ph[2], ph[3]);
                }
                if (!valid) {
#pragma unroll
                    for (int i = 0; i < H; i += 8) ptx::st_shared_v4(p_at(i), 0u, 0u, 0u, 0u);
                }
                const float2 m = __half22float2(top);
                return valid && fmaxf(m.x, m.y) > 32768.f;
            };
            static_assert(kMost == 15.f, "the limit of p above");
            for (int ch = cur.chunk_begin; ch < cur.chunk_end; ch += 2, ++jj) {
                const bool first = ch == cur.chunk_begin;
                const int nh = min(2, cur.chunk_end - ch);
                // Keys of this block, and whether this thread's is one of them.
                const int keys = min(nh * kChunk, L - ch * kChunk);
                const bool valid = key < keys;
                const uint32_t sbuf = jj & 1;
                // The block's scales have landed, P buffer (jj & 1) is free (P.V of
                // block jj - 2 has completed), the scores are there.
                {
                    bool in = ptx::mbar_wait(bar(S::KV_FULL + stage), phase, a.wait_ns);
                    if (jj >= 2)
                        in &= ptx::mbar_wait(bar(S::P_FREE + sbuf), ((jj >> 1) - 1) & 1, a.wait_ns);
                    in &= ptx::mbar_wait(bar(S::S_FULL + sbuf), (jj >> 1) & 1, a.wait_ns);
                    if (!__all_sync(kFull, in)) {
                        fail();
                        ok = false;
                        break;
                    }
                }
                ptx::tc_fence_after();
                const uint8_t* sc = smem + S::OFF_SCALE + stage * 2 * kKeys;
                const int vbyte = sc[kKeys + key];
                const float F = scale_of(sc[key]);
                const float vs = static_cast<float>(vbyte - 127);
                __syncwarp();
                // (the score product has read the keys, this warp their scales)
                if (lane == 0) ptx::mbar_arrive(bar(S::KV_EMPTY + stage));
                if (first && !move_refs(jj, true, valid, F, vs)) {
                    ok = false;
                    break;
                }
                const bool over = probabilities(jj, valid, F, vs);
                ptx::fence_proxy_async_smem();
                if (!first) {
                    // P is handed over only when the warpgroup has found its rows' p in
                    // range (one vote per block but the first of each piece).
                    const bool any = __any_sync(kFull, over);
                    if (lane == 0) {
                        *reinterpret_cast<volatile uint8_t*>(&misc->vote[sbuf][warp]) = any;
                        ptx::mbar_arrive(bar(S::CHECK + wg));
                    }
                    if (!wait_all(bar(S::CHECK + wg), (jj - kk - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (*reinterpret_cast<const uint32_t*>(&misc->vote[sbuf][4 * wg]) != 0) {
                        if (!move_refs(jj, false, valid, F, vs)) {
                            ok = false;
                            break;
                        }
                        (void)probabilities(jj, valid, F, vs);
                        ptx::fence_proxy_async_smem();
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(bar(S::P_FULL + sbuf));
                    ptx::mbar_arrive(bar(S::S_FREE + sbuf));
                }
                if (valid) {
                    const float wkey = inv_scale_of(vbyte);
                    const uint64_t w2 = ptx::f2_pack(wkey, wkey);
#pragma unroll
                    for (int i = 0; i < H; i += 2)
                        ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(x[i], x[i + 1]), w2,
                                                   ptx::f2_pack(l[i], l[i + 1])),
                                       l[i], l[i + 1]);
                }
                if (++stage == S::NS) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            // ---- epilogue: the rows' sums over the key lanes, then O.
            reduce_columns<H>(l, lane, [](float p, float q) { return p + q; });
#pragma unroll
            for (int i = 0; i < (H + 31) / 32; ++i)
                if (i * 32 + lane < H) wmax[quad * R + row0 + i * 32 + lane] = l[i];
            if (!meet()) {
                ok = false;
                break;
            }
            float* slot = a.ws + static_cast<size_t>(cur.slot) * slot_floats(D);
            {
                const int r = threadIdx.x;
                if (r < Mrb) {
                    slot[r] = -nref(r);
                    slot[kRows + r] = (wmax[r] + wmax[R + r]) + (wmax[2 * R + r] + wmax[3 * R + r]);
                }
            }
            if (!wait_all(bar(S::O_FULL), kk & 1)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            // An M = 64 accumulator (D = 64) keeps its rows in the first 16
            // lanes of each warp's 32.
            const int dim = D == 128 ? key : quad * 16 + lane;
            float* acc = slot + 2 * kRows + dim;
#pragma unroll
            for (int c = 0; c < H; c += 8) {
                float o[8];
                ptx::tmem_ld8(lanes + S::TM_O + row0 + c, o);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = row0 + c + i;
                    if (r < Mrb && (D == 128 || lane < 16))
                        acc[static_cast<size_t>(r) * D] = o[i];
                }
            }
            ptx::tc_fence_before();
            // wmax, nref and Q of this segment have been read when all are here
            if (!meet()) {
                ok = false;
                break;
            }
            if (lane == 0) ptx::mbar_arrive(bar(S::O_FREE));
            ++kk;
        }
    }

    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Tree pass and merge.  A CTA takes 4 RW query rows of a unit, a warp RW of them.
//
// Tree pass (reads only this call's inputs, so it runs before the wait for the
// prefix pass): S = Q K^T and O = P V over at most 64 tree tokens with bf16
// mma.sync, whose tile is 16 rows; P enters as two bf16 rows (value and
// remainder), because a row may see only a few tree tokens.  Scores of hidden
// tokens become -inf whatever K holds; a non-finite V value is left out of the
// product and added to the rows that see it.
//
// Merge: a warp reads whole rows of the partials, eight loads of 16 bytes to a lane
// in flight together with the references and sums.  It is bound by round trips:
// with few rows a CTA takes four, so that every warp has one row and its
// partials come in one or two trips.
// ---------------------------------------------------------------------------
constexpr int kTileRows = 16;
constexpr int kMergeCtaWarps = 4;
constexpr int kMergeThreads = 32 * kMergeCtaWarps;

struct TreeMergeArgs {
    const uint16_t* q;
    const uint16_t* tree_k;
    const uint16_t* tree_v;
    const uint64_t* mask;
    int mask_stride;
    const int32_t* parents;
    int parents_stride;
    uint64_t* mask_out;
    const int32_t* seq_lens;
    const float* ws;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int B, Hq, Hkv, G, T, M, RB, P, max_pages, n_ctas, ovh;
    float scale_log2;
};

// D += A B for one 16 x 8 tile, 16 deep, bf16 in, fp32 out.
__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Ancestor-or-self bits of nodes lane and lane + 32 by following parents six
// doublings deep; an invalid parent makes its node a root and is told of.
__device__ bool ancestor_bits(const int32_t* parents, int T, int lane, uint64_t bits[2]) {
    int jump[2];
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        int p = i < T ? parents[i] : -1;
        if (p < -1 || p >= i) {
            bad = bad || i < T;
            p = -1;
        }
        jump[h] = p;
        bits[h] = i < T ? 1ull << i : 0ull;
    }
#pragma unroll
    for (int round = 0; round < 6; ++round) {
        uint64_t nb[2];
        int nj[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = max(jump[h], 0);
            const uint64_t b0 = __shfl_sync(kFull, bits[0], j & 31);
            const uint64_t b1 = __shfl_sync(kFull, bits[1], j & 31);
            const int j0 = __shfl_sync(kFull, jump[0], j & 31);
            const int j1 = __shfl_sync(kFull, jump[1], j & 31);
            const bool on = jump[h] >= 0;
            nb[h] = on ? bits[h] | (j < 32 ? b0 : b1) : bits[h];
            nj[h] = on ? (j < 32 ? j0 : j1) : -1;
        }
        bits[0] = nb[0];
        bits[1] = nb[1];
        jump[0] = nj[0];
        jump[1] = nj[1];
    }
    return __any_sync(kFull, bad);
}

// A pair of bf16 halves with those that are not finite set to zero.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

template <int D, int RW>
__global__ void __launch_bounds__(kMergeThreads, 6) tree_merge_fp8_kernel(const TreeMergeArgs a) {
    constexpr int ROWS = RW * kMergeCtaWarps;  // of this CTA: 4 or 16
    constexpr int NT = D / 8 / kMergeCtaWarps;  // 8-wide accumulator tiles of a warp
    __shared__ float s_score[kTileRows][TREE_ATTN_MAX_T + 4];  // then P, hi | lo << 16
    __shared__ uint64_t s_bits[TREE_ATTN_MAX_T];
    __shared__ float s_m[ROWS], s_l[ROWS];  // the tree's share: reference, sum,
    __shared__ __align__(16) float s_o[ROWS][D + 4];  // accumulator
    __shared__ int s_first, s_count, s_all;
    __shared__ uint32_t s_has;  // which of the first 32 partials there are
    __shared__ long long s_W;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x;
    const int rb = unit % a.RB;
    const int hk = (unit / a.RB) % a.Hkv;
    const int b = unit / (a.RB * a.Hkv);
    const int r0 = blockIdx.y * ROWS;  // first row of the row block taken here
    // The next kernel waits for this grid before it writes anything read here.
    ptx::grid_dep_launch();

    auto row_at = [&](int r) -> int { return rb * kRows + r0 + r; };  // row of the unit
    auto row_ok = [&](int r) -> bool { return merge_has_row(rb, r0, r, ROWS, a.M); };
    // Element offset in q and out of the d values of row rr of the unit; lse has
    // one per d.
    auto row_offset = [&](int rr) -> long long {
        return ((static_cast<long long>(b) * a.T + rr / a.G) * a.Hq + hk * a.G + rr % a.G) * D;
    };
    auto q_row = [&](int r) -> const uint16_t* {
        return a.q + row_offset(merge_reads_row(rb, r0, r, ROWS, a.M));
    };
    const int g = lane >> 2, t = lane & 3;  // lane of an accumulator: rows g, g + 8

    // ---- tree scores: 16 tokens to a warp
    {
        const int key0 = warp * 16;
        float c[2][4] = {};
        if (key0 < a.T) {
            // A lane holds eight consecutive elements of rows g and g + 8 and of
            // token g of each 8-token tile: a dot product does not mind which of
            // the 16 places of a step an element takes.
            const uint16_t* q0 = q_row(g) + t * 8;
            const uint16_t* q1 = q_row(g + 8) + t * 8;
            auto token = [&](int j) -> const uint16_t* {
                return a.tree_k +
                       ((static_cast<long long>(b) * a.T + min(j, a.T - 1)) * a.Hkv + hk) * D +
                       t * 8;
            };
            const uint16_t* k0 = token(key0 + g);
            const uint16_t* k1 = token(key0 + 8 + g);
            uint4 x[4][D / 32];
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                x[0][s] = __ldg(reinterpret_cast<const uint4*>(q0 + s * 32));
                x[1][s] = __ldg(reinterpret_cast<const uint4*>(q1 + s * 32));
                x[2][s] = __ldg(reinterpret_cast<const uint4*>(k0 + s * 32));
                x[3][s] = __ldg(reinterpret_cast<const uint4*>(k1 + s * 32));
            }
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                const uint32_t a0[4] = {x[0][s].x, x[1][s].x, x[0][s].y, x[1][s].y};
                const uint32_t a1[4] = {x[0][s].z, x[1][s].z, x[0][s].w, x[1][s].w};
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma_16816(c[n], a0, x[2 + n][s].x, x[2 + n][s].y);
                    mma_16816(c[n], a1, x[2 + n][s].z, x[2 + n][s].w);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s_score[g + 8 * (i >> 1)][key0 + 8 * n + 2 * t + (i & 1)] = c[n][i] * a.scale_log2;
    }
    // ---- masks (warp 3: the one least likely to have had tokens)
    if (warp == 3) {
        uint64_t bits[2] = {0ull, 0ull};
        if (a.parents != nullptr) {
            const bool bad = ancestor_bits(
                a.parents + static_cast<size_t>(b) * a.parents_stride, a.T, lane, bits);
            // One CTA per tree reports and writes the masks out.
            const bool writer = unit == b * a.Hkv * a.RB && blockIdx.y == 0 &&
                                (a.parents_stride != 0 || b == 0);
            if (writer && bad && lane == 0) report(a.status, TREE_ATTN_STATUS_BAD_PARENT);
            if (writer && a.mask_out != nullptr) {
                uint64_t* mo = a.mask_out + static_cast<size_t>(b) * a.parents_stride;
                if (lane < a.T) mo[lane] = bits[0];
                if (lane + 32 < a.T) mo[lane + 32] = bits[1];
            }
        } else {
            const uint64_t live = a.T < 64 ? (1ull << a.T) - 1ull : ~0ull;
            const uint64_t* m = a.mask + static_cast<size_t>(b) * a.mask_stride;
            if (lane < a.T) bits[0] = m[lane] & live;
            if (lane + 32 < a.T) bits[1] = m[lane + 32] & live;
        }
        s_bits[lane] = bits[0];
        s_bits[lane + 32] = bits[1];
    }
    // ---- the prefix CTAs that hold this unit's partials (warp 2): s_first and the
    // s_count - 1 behind it
    if (warp == 2) {
        long long W = 0, base = 0;
        int nch = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int bi = b0 + lane;
            bool bad;
            const int n =
                bi < a.B ? unit_chunks(a.seq_lens[bi], a.P, a.max_pages, kTreeNone, 0, bad) : 0;
            const int len = unit_len(n, a.ovh);
            W += __reduce_add_sync(kFull, len);
            base += __reduce_add_sync(kFull, bi < b ? len : 0);
            nch += __reduce_add_sync(kFull, bi == b ? n : 0);
        }
        const int upb = a.Hkv * a.RB;
        W *= upb;
        base *= upb;
        int first = 0, count = 0;
        if (nch > 0) {
            const long long start =
                base + static_cast<long long>(unit - b * upb) * unit_len(nch, a.ovh);
            first = cta_of(start, W, a.n_ctas);
            count = cta_of(start + nch - 1, W, a.n_ctas) - first + 1;
        }
        // With a step or more to every CTA each of them has a partial.
        const bool all = W >= a.n_ctas;
        const uint32_t some = __ballot_sync(
            kFull, lane < count && (all || cta_has_work(first + lane, W, a.n_ctas)));
        if (lane == 0) {
            s_first = first;
            s_count = count;
            s_all = all;
            s_has = some;
            s_W = W;
        }
    }
    __syncthreads();

    // ---- softmax of the tree scores, RW rows to a warp (the tile's other rows are
    // never looked at)
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int r = warp * RW + i;
        const uint64_t bits = row_ok(r) ? s_bits[row_at(r) / a.G] : 0ull;
        const bool see0 = (bits >> lane) & 1ull, see1 = (bits >> (lane + 32)) & 1ull;
        const float x0 = see0 ? s_score[r][lane] : kNegInf;
        const float x1 = see1 ? s_score[r][lane + 32] : kNegInf;
        float m = fmaxf(x0, x1);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        const float ref = m == kNegInf ? 0.f : m;
        const float p0 = see0 ? ptx::ex2(x0 - ref) : 0.f;
        const float p1 = see1 ? ptx::ex2(x1 - ref) : 0.f;
        float l = p0 + p1;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
        if (lane == 0) {
            // (a row of NaN scores has no largest; its sum is NaN all the same)
            s_m[r] = bits != 0 && m == kNegInf ? 0.f : m;
            s_l[r] = l;
        }
        auto split = [](float p) -> float {
            const uint32_t hi = pack_bf16(p, 0.f) & 0xffffu;
            const uint32_t lo = pack_bf16(p - __uint_as_float(hi << 16), 0.f) & 0xffffu;
            return __uint_as_float(hi | (lo << 16));
        };
        s_score[r][lane] = split(p0);
        s_score[r][lane + 32] = split(p1);
    }
    __syncthreads();

    // ---- O = P V: this thread's dimensions are dim .. dim + 2 NT - 1.  Column c of
    // tile n stands for dimension dim0 + NT c + n, so that a lane's B elements of all
    // tiles (columns g) and its accumulator's (columns 2t, 2t + 1) lie side by side.
    {
    const int dim0 = warp * NT * 8;
    const int dim = dim0 + 2 * t * NT;
    float o[NT][4] = {};
    {
        const uint16_t* v0 = a.tree_v + (static_cast<long long>(b) * a.T * a.Hkv + hk) * D;
        const long long vs = static_cast<long long>(a.Hkv) * D;  // from token to token
        bool odd = false;  // a value that is not finite
        static_assert(NT == 4 || NT == 2, "columns of a lane");
        constexpr int NW = NT / 2;  // 32-bit words of a lane's NT columns
#pragma unroll 2
        for (int k0 = 0; k0 < a.T; k0 += 16) {
            uint32_t vw[4][NW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = min(k0 + 2 * t + (i & 1) + 8 * (i >> 1), a.T - 1);
                const uint16_t* p = v0 + j * vs + dim0 + NT * g;
                if constexpr (NT == 4) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
                    vw[i][0] = w.x;
                    vw[i][NW - 1] = w.y;
                } else {
                    vw[i][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
                }
            }
            bool here = false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    here |= (((vw[i][w] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u) != 0;
            if (__any_sync(kFull, here)) {
                odd = true;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < NW; ++w) vw[i][w] = finite_pair(vw[i][w]);
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = g + 8 * (i & 1), k = k0 + 2 * t + 8 * (i >> 1);
                const uint32_t u0 = __float_as_uint(s_score[r][k]);
                const uint32_t u1 = __float_as_uint(s_score[r][k + 1]);
                hi[i] = __byte_perm(u0, u1, 0x5410);
                lo[i] = __byte_perm(u0, u1, 0x7632);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t pick_half = n & 1 ? 0x7632 : 0x5410;
                const uint32_t b0 = __byte_perm(vw[0][n / 2], vw[1][n / 2], pick_half);
                const uint32_t b1 = __byte_perm(vw[2][n / 2], vw[3][n / 2], pick_half);
                mma_16816(o[n], hi, b0, b1);
                mma_16816(o[n], lo, b0, b1);
            }
        }
        if (odd) {
#pragma unroll 1
            for (int j = 0; j < a.T; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = g + 8 * (i >> 1);
                        const uint32_t v = __ldg(v0 + j * vs + dim + (i & 1) * NT + n);
                        if ((v & 0x7f80u) == 0x7f80u && row_ok(r) &&
                            ((s_bits[row_at(r) / a.G] >> j) & 1ull))
                            o[n][i] += __uint_as_float(v << 16);
                    }
        }
    }

#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i;
            if (r >= ROWS) continue;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                s_o[r][dim + n] = o[n][2 * i];
                s_o[r][dim + NT + n] = o[n][2 * i + 1];
            }
        }
    }
    __syncthreads();

    // ---- merge with the prefix pass's partials (read through L2: the prefix grid
    // writes them while this one is resident)
    ptx::grid_dep_wait();
    constexpr int E = D / 32;    // dimensions of a lane
    constexpr int PF = 8 / RW;   // partials of a row in flight
    const int count = s_count;
    const uint32_t some = s_has;
    const size_t sf = static_cast<size_t>(slot_floats(D));
    const float* slots = a.ws + static_cast<size_t>(unit + s_first) * sf;
    auto has = [&](int v) -> bool {
        if (v < 32) return (some >> v) & 1u;
        return v < count && (s_all || cta_has_work(s_first + v, s_W, a.n_ctas));
    };
    // E accumulator values of row r in partial v; a partial that is not there has
    // weight 0 and is read as slot 0, so that no branch stands between loads.
    auto fetch = [&](int v, int r, float* x) {
        const float* p = slots + static_cast<size_t>(has(v) ? v : 0) * sf + 2 * kRows +
                         static_cast<size_t>(r) * D + lane * E;
        if constexpr (E == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(p));
            x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
        } else {
            const float2 f = __ldcg(reinterpret_cast<const float2*>(p));
            x[0] = f.x, x[1] = f.y;
        }
    };
    int at[RW];  // rows of the slots; a row that is not there reads the first
    bool live[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        live[i] = row_ok(warp * RW + i);
        at[i] = r0 + (live[i] ? warp * RW + i : 0);
    }
    float x[RW][PF][E], m[RW], l[RW];
    if (count > 0) {
        // One round trip: references and sums (lane v: partial v) and the first
        // partials' accumulators.
        const float* mine = slots + static_cast<size_t>(has(lane) ? lane : 0) * sf;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            m[i] = __ldcg(mine + at[i]);
            l[i] = __ldcg(mine + kRows + at[i]);
        }
#pragma unroll
        for (int k = 0; k < PF; ++k)
#pragma unroll
            for (int i = 0; i < RW; ++i) fetch(k, at[i], x[i][k]);
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int r = warp * RW + i;
        if (count == 0 || !has(lane)) {
            m[i] = kNegInf;
            l[i] = 0.f;
        }
        float top = m[i];
        for (int v0 = 32; v0 < count; v0 += 32)  // (rare)
            if (has(v0 + lane))
                top = fmaxf(top, __ldcg(slots + static_cast<size_t>(v0 + lane) * sf + at[i]));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        top = fmaxf(top, s_m[r]);
        const float ref = top == kNegInf ? 0.f : top;
        float w = ptx::ex2(m[i] - ref);  // lane v: weight of partial v
        float sum = m[i] == kNegInf ? 0.f : w * l[i];
        const float ws = ptx::ex2(s_m[r] - ref);
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = ws * s_o[r][lane * E + e];
        for (int v0 = 0; v0 < count; v0 += 32) {
            if (v0 > 0) {
                float lv = 0.f;
                w = 0.f;
                if (has(v0 + lane)) {
                    const float* p = slots + static_cast<size_t>(v0 + lane) * sf + at[i];
                    w = ptx::ex2(__ldcg(p) - ref);
                    lv = __ldcg(p + kRows);
                }
                sum = fmaf(w, lv, sum);
            }
            const int here = min(32, count - v0);
            for (int k0 = 0; k0 < here; k0 += PF) {
                if (v0 + k0 > 0) {
#pragma unroll
                    for (int k = 0; k < PF; ++k) fetch(v0 + k0 + k, at[i], x[i][k]);
                }
#pragma unroll
                for (int k = 0; k < PF; ++k) {
                    const float wk = __shfl_sync(kFull, w, (k0 + k) & 31);
                    if (k0 + k >= here) continue;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = fmaf(wk, x[i][k][e], o[e]);
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
        sum = fmaf(ws, s_l[r], sum);
        if (!live[i]) continue;
        const bool none = top == kNegInf;  // no key at all
        const float inv = none ? 0.f : 1.f / sum;
        const long long to = row_offset(row_at(r));
        uint32_t word[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2)
            word[e / 2] = none ? 0u : pack_bf16(o[e] * inv, o[e + 1] * inv);
        uint16_t* dst = a.out + to + lane * E;
        if constexpr (E == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(word[0], word[1]);
        else
            *reinterpret_cast<uint32_t*>(dst) = word[0];
        if (lane == 0) a.lse[to / D] = none ? kNegInf : (top + log2f(sum)) * kLn2;
    }
}

// Four rows to a CTA as long as all CTAs run at once (six to an SM), else sixteen:
// the tree's scores are then made for fewer CTAs.
template <int D>
cudaError_t launch_tree_merge(const TreeMergeArgs& v, int units, int sms, cudaStream_t stream) {
    const unsigned fours = static_cast<unsigned>(merge_groups(v.M, 4));
    if (static_cast<long long>(units) * fours <= 6LL * sms)
        return launch_dependent(tree_merge_fp8_kernel<D, 1>,
                                dim3(static_cast<unsigned>(units), fours), dim3(kMergeThreads), 0,
                                stream, v);
    return launch_dependent(
        tree_merge_fp8_kernel<D, 4>,
        dim3(static_cast<unsigned>(units), static_cast<unsigned>(merge_groups(v.M, 16))),
        dim3(kMergeThreads), 0, stream, v);
}

template <int D, int R, int WG>
cudaError_t launch_prefix_fp8(const Fp8Args& a, const CUtensorMap& tk, const CUtensorMap& tv,
                              int dev, cudaStream_t stream) {
    using S = Shape<D, R, WG>;
    // Devices on which the shared-memory opt-in has been applied.
    static std::atomic<unsigned long long> configured{0};
    const unsigned long long bit = 1ull << (dev & 63);
    if ((configured.load() & bit) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(
            prefix_fp8_kernel<D, R, WG>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return launch_dependent(prefix_fp8_kernel<D, R, WG>, dim3(a.n_ctas), dim3(S::THREADS), S::SMEM,
                            stream, tk, tv, a);
}

// The smallest tile that holds a unit's rows: every lane of the softmax works
// on each of them, so idle rows cost as much as used ones.  8 x 16384 tokens, 8 KV
// heads, d = 128: 16 rows 52 us, 32: 60, 48: 66, 64: 80, 80: 98, 128: 137.  (Other
// numbers of warpgroups, measured with P in two 8-bit halves: two for 48 rows 60 us
// for 59, two for 64 rows 75 for 72, four for 32 rows 53 for 52; five for 80 rows 3 %
// slower.)
template <int D>
cudaError_t launch_prefix_fp8_rows(const Fp8Args& a, const CUtensorMap& tk,
                                   const CUtensorMap& tv, int dev, cudaStream_t stream) {
    const int rows = a.M < kRows ? a.M : kRows;
    if (rows <= 16) return launch_prefix_fp8<D, 16, 2>(a, tk, tv, dev, stream);
    if (rows <= 32) return launch_prefix_fp8<D, 32, 2>(a, tk, tv, dev, stream);
    if (rows <= 48) return launch_prefix_fp8<D, 48, 3>(a, tk, tv, dev, stream);
    if (rows <= 64) return launch_prefix_fp8<D, 64, 4>(a, tk, tv, dev, stream);
    if (rows <= 80) return launch_prefix_fp8<D, 80, 2>(a, tk, tv, dev, stream);
    return launch_prefix_fp8<D, 128, 2>(a, tk, tv, dev, stream);
}

// The [num_pages * Hkv * P][d] codes of a pool in boxes of up to 64 tokens.
bool encode_codes(CUtensorMap* map, const void* base, long long rows, int d, int P) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(d),
                               static_cast<cuuint32_t>(P < kChunk ? P : kChunk)};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                        d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" int tree_attn_verify_fp8(
    const uint16_t* q, const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_scales,
    const uint8_t* v_scales, const int32_t* block_table, int max_pages_per_seq,
    const int32_t* seq_lens, const uint16_t* tree_k, const uint16_t* tree_v, const uint64_t* mask,
    int mask_stride, const int32_t* parents, int parents_stride, uint64_t* mask_out,
    uint16_t* out, float* lse, int B, int Hq, int Hkv, int d, int T, int page_size, int num_pages,
    float softmax_scale, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    if (B < 0 || T < 1 || T > TREE_ATTN_MAX_T || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 ||
        (d != 64 && d != 128) || !page_size_ok(page_size) || max_pages_per_seq < 1 ||
        num_pages < 1 || static_cast<long long>(num_pages) * Hkv * page_size >= (1LL << 31) ||
        !std::isfinite(softmax_scale) || (mask_stride != 0 && mask_stride != T) ||
        (parents_stride != 0 && parents_stride != T) || (mask != nullptr && parents != nullptr))
        return TREE_ATTN_ERR_SHAPE;
    if (B == 0) return TREE_ATTN_OK;
    if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !seq_lens ||
        !tree_k || !tree_v || (!mask && !parents) || !out || !lse)
        return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(q, 16) || !ptr_aligned(k_pages, 16) || !ptr_aligned(v_pages, 16) ||
        !ptr_aligned(k_scales, 16) || !ptr_aligned(v_scales, 16) || !ptr_aligned(tree_k, 16) ||
        !ptr_aligned(tree_v, 16) || !ptr_aligned(out, 16) || !ptr_aligned(block_table, 4) ||
        !ptr_aligned(seq_lens, 4) || !ptr_aligned(lse, 4) || !ptr_aligned(mask, 8) ||
        !ptr_aligned(parents, 4) || !ptr_aligned(mask_out, 8) || !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    const size_t need = tree_attn_workspace_size(B, Hq, Hkv, d, T, 0, page_size);
    if (need == 0) return TREE_ATTN_ERR_CUDA;
    if (workspace == nullptr || !ptr_aligned(workspace, 256) || workspace_bytes < need)
        return TREE_ATTN_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return TREE_ATTN_ERR_CUDA;
    const Plan plan = make_plan(B, Hq, Hkv, T, page_size, max_pages_per_seq, sms, 0, kTreeNone);
    const long long rows = static_cast<long long>(num_pages) * Hkv * page_size;
    CUtensorMap tk, tv;
    if (!encode_codes(&tk, k_pages, rows, d, page_size) ||
        !encode_codes(&tv, v_pages, rows, d, page_size))
        return TREE_ATTN_ERR_CUDA;
    Fp8Args a;
    a.q = q;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.ws = static_cast<float*>(workspace);
    a.status = status;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = plan.G;
    a.T = T;
    a.M = plan.M;
    a.RB = plan.RB;
    a.P = page_size;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.n_ctas = plan.n_ctas;
    a.ovh = kOverhead;
    a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
    a.wait_ns = wait_limit_ns();
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((d == 128 ? launch_prefix_fp8_rows<128>(a, tk, tv, dev, st)
                  : launch_prefix_fp8_rows<64>(a, tk, tv, dev, st)) != cudaSuccess)
        return TREE_ATTN_ERR_CUDA;
    TreeMergeArgs v;
    v.q = q;
    v.tree_k = tree_k;
    v.tree_v = tree_v;
    v.mask = mask;
    v.mask_stride = mask_stride;
    v.parents = parents;
    v.parents_stride = parents_stride;
    v.mask_out = mask_out;
    v.seq_lens = seq_lens;
    v.ws = a.ws;
    v.out = out;
    v.lse = lse;
    v.status = status;
    v.B = B;
    v.Hq = Hq;
    v.Hkv = Hkv;
    v.G = a.G;
    v.T = T;
    v.M = a.M;
    v.RB = a.RB;
    v.P = page_size;
    v.max_pages = max_pages_per_seq;
    v.n_ctas = a.n_ctas;
    v.ovh = a.ovh;
    v.scale_log2 = a.scale_log2;
    const cudaError_t e = d == 128 ? launch_tree_merge<128>(v, plan.units, sms, st)
                                   : launch_tree_merge<64>(v, plan.units, sms, st);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
