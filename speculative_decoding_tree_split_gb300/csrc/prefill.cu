// prefill.cu -- causal attention over whole prompts of different lengths,
// packed one after the other, with grouped heads.
//
// For token i of a sequence and a query head: out = sum_{j <= i} p_j v_j / l,
// p_j = 2^(c <q, k_j> - m), l = sum_j p_j, c = softmax scale * log2(e), m a
// reference near the row's maximum.  One pass over the keys, 2 * d * 2
// operations per (row, key): bound by the tensor cores for long prompts.
//
// * A unit is (sequence, KV head, 256 consecutive rows), row = token * G + head
//   of the group, so any number of heads to a KV head fills the tiles and all
//   of them share the K/V tiles.  Its rows are two tiles of 128.
// * One warp issues the MMAs of both tiles in turn: while tile A's softmax
//   works on its scores, the tensor cores run O += P V and the next S = Q K^T
//   of tile B, and the other way round.
// * One thread per row: 128 scores from TMEM, maximum, exponentials, P back to
//   TMEM over its own scores.  The reference moves only when a maximum exceeds
//   it by 8 binades, so O is seldom rescaled.
// * P is bf16 because V is: an MMA's operands have one type, and fp16 does not hold
//   every V.  The row's sum takes p in fp32, so that lse has all its bits; a
//   row whose probabilities all round the same way is then off by half a bf16 step
//   (2^-8 of it at the most), as in the pass over the bf16 cache.
// * Keys a row may not see get a score of -inf by index, whatever K holds.
//   V of such keys still meets P = 0 in the tensor cores, and 0 * NaN is not 0:
//   in blocks that some row does not see whole, two warps clear the non-finite
//   values of the V tile, and the epilogue adds them to the rows that see them.
// * The grid is one CTA per unit, longest first, but a CTA that has started goes
//   on with units whose CTAs have not (cluster launch control): their loads
//   and queries are under way while the unit before ends.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/tree_attn.h"
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
constexpr int kKeys = 128;           // keys of a block
constexpr int kUnit = 2 * kRows;     // rows of a unit
// Keys of a block whose probabilities are handed over before the rest (16384 tokens,
// 32 heads: 32 keys 1457 us, 64 keys 1439 us, 96 keys 1463 us).
constexpr int kFirstKeys = 64;
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpClean = 10;
constexpr int kThreads = 384;        // two softmax warpgroups and one of helpers

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

struct PrefillArgs {
    const uint16_t* q;
    const uint16_t* v;
    long long q_ts, q_hs, v_ts, v_hs;  // token and head strides (elements)
    int k_heads, v_heads;  // 0: one head stands for all (stride 0)
    int q_tiles, o_tiles;  // queries (results) move as boxes of the tensor maps
    const int32_t* cu;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int B, N, Hq, Hkv, G;
    float scale_log2;      // > 0
    float inv_g;           // 1 / G
    uint32_t q_sign;       // flips the queries' signs where the scale is negative
    uint32_t q_keep;       // 0 clears the queries (scale 0)
    unsigned long long wait_ns;
};

template <int D>
struct Shape {
    static constexpr int DH = D / 64;              // 128-byte columns of d
    static constexpr int Q_TILE = kRows * D * 2;   // one tile's queries
    static constexpr int Q_ATOM = kRows * 128;
    static constexpr int TILE = kKeys * D * 2;     // K or V of one block
    static constexpr int ATOM = kKeys * 128;
    static constexpr int NS = D == 128 ? 4 : 8;    // ring slots, K and V in turn
    // Registers: 168 a thread at launch; the helpers give theirs to the softmax, which
    // holds a row's 128 scores.  The split leaves neither side with spills (114 bytes
    // in the copies' warp cost a ragged batch 20 %).
    static constexpr int SOFT_REGS = 232, HELP_REGS = 40;
    static_assert(256 * SOFT_REGS + 128 * HELP_REGS <= kThreads * 168, "registers at launch");
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + 2 * Q_TILE;
    static constexpr int OFF_OUT = OFF_RING + NS * TILE;  // [8 warps][32 rows][64 columns]
    static constexpr int OFF_MISC = OFF_OUT + 8 * 32 * 128;
    static constexpr int OFF_BAR = OFF_MISC + 192;
    static constexpr int FULL = 0;
    static constexpr int EMPTY = NS;
    static constexpr int S_FULL = 2 * NS;      // [2] by tile
    static constexpr int P_FULL = S_FULL + 2;  // [2]: all of P
    static constexpr int O_FULL = S_FULL + 4;  // [2]
    static constexpr int Q_FULL = S_FULL + 6;  // [2]
    static constexpr int ASK = S_FULL + 8;    // V of an edge block has landed: clean it
    static constexpr int CLEAN = S_FULL + 9;  // it is clean
    static constexpr int P_HALF = S_FULL + 10;  // [2]: P of the first keys
    static constexpr int UNIT_FULL = S_FULL + 12;   // [2]: a unit has been announced
    static constexpr int UNIT_EMPTY = S_FULL + 14;  // [2]: every warp has read it
    static constexpr int ANSWER = S_FULL + 16;      // the launch control has answered
    static constexpr int DRAIN = S_FULL + 17;
    static constexpr int Q_FREE = S_FULL + 18;  // [2]: a unit's last scores have been made
    static constexpr int NBAR = S_FULL + 20;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 1024;  // + alignment slack
    // TMEM: S of both tiles (P over them), then O of both.
    static constexpr int TM_S = 0;
    static constexpr int TM_O = 2 * kKeys;
    static_assert(TM_O + 2 * D <= 512, "TMEM budget");
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
    static_assert(SMEM > 114 * 1024, "one CTA per SM keeps TMEM allocation uncontended");
};

// Row r of a sequence is token r / G, head r % G of the group (N * G < 2^31: the
// host checks).
struct Unit {
    int first, len;  // packed rows of the sequence
    int hk, rb;      // KV head; row block, -1: no more units
    int tok0, rem0;  // token and head of its first row
    int nA, nB;      // blocks of its two tiles: they end with the last row's token
};

struct Misc {
    ulonglong2 answer;  // of the launch control
    Unit unit[2];       // announced units, in turn
    uint32_t tmem_base;
    int abort;
    uint32_t q_loads;   // query tiles that the copies' warp has loaded
    int dirty[4][2];    // by unit, in turn, and cleaning warp: V held something
};
static_assert(sizeof(Misc) <= 192, "Misc fits its slot");
constexpr int kReaders = 11;  // warps that read announced units: all but the copies'

// n / G for n < 2^17: (n + 1/2) / G is at least 1 / (2 G) away from an integer, and
// its two roundings move it by less than (n + 1/2) / G * 2^-22.
__device__ __forceinline__ int by_group(const PrefillArgs& a, int n) {
    return static_cast<int>((static_cast<float>(n) + 0.5f) * a.inv_g);
}

// Row blocks of sequence b (0 where its range is out of order or empty).
__device__ __forceinline__ int row_blocks(const PrefillArgs& a, int b) {
    if (b >= a.B) return 0;
    const int lo = a.cu[b], hi = a.cu[b + 1];
    if (lo < 0 || hi < lo || hi > a.N) return 0;
    const long long rows = static_cast<long long>(hi - lo) * a.G;
    return static_cast<int>((rows + kUnit - 1) / kUnit);
}

// Unit `index` in the order of falling row-block index (so of falling work), KV
// heads innermost; rb = -1 past the last.  One warp, every lane gets it.  With
// n_b row blocks in sequence b, the units of index >= r number
// sum_b max(0, n_b - r), so the index of unit u is found by halving.
__device__ Unit find_unit(const PrefillArgs& a, int lane, int index) {
    const int id = index / a.Hkv;
    Unit u;
    u.hk = index % a.Hkv;
    u.rb = -1;
    u.first = u.len = u.tok0 = u.rem0 = u.nA = u.nB = 0;
    const int n0 = row_blocks(a, lane);  // the first 32 sequences stay here
    auto count = [&](int r) -> int {
        int n = max(0, n0 - r);
        for (int b = 32; b < a.B; b += 32) n += max(0, row_blocks(a, b + lane) - r);
        return __reduce_add_sync(kFull, n);
    };
    if (id >= count(0)) return u;
    int lo = 0, hi = n0;  // the largest r with count(r) > id
    for (int b = 32; b < a.B; b += 32) hi = max(hi, row_blocks(a, b + lane));
    hi = __reduce_max_sync(kFull, hi);
    if (a.B == 1) lo = hi - 1 - id;
    else
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (count(mid) > id)
                lo = mid;
            else
                hi = mid;
        }
    u.rb = lo;
    int rest = id - count(lo + 1);  // which of the sequences with n_b > lo
    for (int b = 0; b < a.B; b += 32) {
        const int n = b == 0 ? n0 : row_blocks(a, b + lane);
        const unsigned m = __ballot_sync(kFull, n > lo);
        const int c = __popc(m);
        if (rest < c) {
            const int at = __fns(m, 0, rest + 1);
            u.first = a.cu[b + at];
            u.len = a.cu[b + at + 1] - u.first;
            const int left = u.len * a.G - u.rb * kUnit;  // rows from the first on
            u.tok0 = u.rb * kUnit / a.G;
            u.rem0 = u.rb * kUnit - u.tok0 * a.G;
            auto blocks = [&](int n) -> int {  // for the first n rows
                return (u.tok0 + by_group(a, u.rem0 + min(n, left) - 1)) / kKeys + 1;
            };
            u.nA = blocks(kRows);
            u.nB = left > kRows ? blocks(kUnit) : 0;
            return u;
        }
        rest -= c;
    }
    u.rb = -1;
    return u;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_o, const PrefillArgs a) {
    using S = Shape<D>;
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
            ptx::mbar_init(bar(S::FULL + s), 1);
            ptx::mbar_init(bar(S::EMPTY + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(S::S_FULL + i), 1);
            ptx::mbar_init(bar(S::P_FULL + i), 4);
            ptx::mbar_init(bar(S::P_HALF + i), 4);
            ptx::mbar_init(bar(S::O_FULL + i), 1);
            ptx::mbar_init(bar(S::Q_FULL + i), a.q_tiles ? 1 : 4);
            ptx::mbar_init(bar(S::Q_FREE + i), 1);
        }
        ptx::mbar_init(bar(S::ASK), 1);
        ptx::mbar_init(bar(S::CLEAN), 2);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(S::UNIT_FULL + i), 1);
            ptx::mbar_init(bar(S::UNIT_EMPTY + i), kReaders);
        }
        ptx::mbar_init(bar(S::ANSWER), 1);
        ptx::mbar_init(bar(S::DRAIN), 1);
        misc->abort = 0;
        misc->q_loads = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(ptx::smem_u32(&misc->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc->tmem_base;
    auto fail = [&]() {
        *abort_flag = 1;
        report(a.status, TREE_ATTN_STATUS_TIMEOUT);
    };

    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += kThreads)
            if (a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.N)
                report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);

    // Blocks from `edge` on hold keys that some row of the unit does not see.
    struct Span {
        int nA, nB, n, edge;
    };
    auto span_of = [&](const Unit& u) -> Span {
        return {u.nA, u.nB, max(u.nA, u.nB), (u.tok0 + 1) / kKeys};
    };
    auto wait = [&](int i, uint32_t parity) -> bool {
        const bool all = __all_sync(kFull, ptx::mbar_wait(bar(i), parity & 1, a.wait_ns));
        if (!all) fail();
        return all;
    };
    // Announced unit number k (every warp but the copies' reads each in turn);
    // false: no more, or a wait ran out.
    auto next_unit = [&](uint32_t k, Unit& u) -> bool {
        if (!wait(S::UNIT_FULL + (k & 1), k >> 1)) return false;
        u = misc->unit[k & 1];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(S::UNIT_EMPTY + (k & 1)));
        return u.rb >= 0;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::HELP_REGS));
        if (warp == kWarpTma) {
            // ================= units and copies: K0, V0, K1, V1, ... of each
            Unit u = find_unit(a, lane, blockIdx.x);
            if (lane == 0) {
                misc->unit[0] = u;
                ptx::mbar_arrive(bar(S::UNIT_FULL));
            }
            __syncwarp();
            uint32_t t = 0;  // tiles loaded so far
            bool ok = true;
#pragma unroll 1
            for (uint32_t k = 0; u.rb >= 0; ++k) {
                // One unit ahead: the answer comes in while this one is loaded.
                if (lane == 0) {
                    ptx::fence_proxy_async_smem();  // the last answer has been read
                    ptx::mbar_arrive_expect_tx(bar(S::ANSWER), 16);
                    ptx::try_cancel(ptx::smem_u32(&misc->answer), bar(S::ANSWER));
                }
                __syncwarp();
                // A ring's worth of tiles first, then the next unit is looked up and
                // announced, then the rest.
                const int n2 = 2 * span_of(u).n;
                const int hk_k = a.k_heads ? u.hk : 0, hk_v = a.v_heads ? u.hk : 0;
                auto load = [&](int from, int to) -> bool {
                    if (lane == 0) {
#pragma unroll 1
                        for (int i = from; i < to; ++i, ++t) {
                            const uint32_t s = t % S::NS;
                            if (t >= S::NS && !ptx::mbar_wait(bar(S::EMPTY + s),
                                                              (t / S::NS - 1) & 1, a.wait_ns)) {
                                fail();
                                ok = false;
                                break;
                            }
                            if (*abort_flag) {
                                ok = false;
                                break;
                            }
                            const bool is_v = i & 1;
                            const int tok = u.first + (i >> 1) * kKeys;
                            const uint32_t dst = sb + S::OFF_RING + s * S::TILE;
                            ptx::mbar_arrive_expect_tx(bar(S::FULL + s), S::TILE);
#pragma unroll
                            for (int h = 0; h < S::DH; ++h)
                                ptx::tma_load_3d_keep(dst + h * S::ATOM, is_v ? &tm_v : &tm_k,
                                                      h * 64, is_v ? hk_v : hk_k, tok,
                                                      bar(S::FULL + s));
                        }
                    }
                    ok = __shfl_sync(kFull, ok, 0);
                    return ok;
                };
                // Queries as boxes, once the unit before has made its last scores: of the
                // tiles that the ring has room for by then, the last two are behind them.
                auto queries = [&]() -> bool {
                    if (lane == 0 && a.q_tiles) {
#pragma unroll 1
                        for (int x = 0; x < 2; ++x) {
                            if (k > 0 &&
                                !ptx::mbar_wait(bar(S::Q_FREE + x), (k - 1) & 1, a.wait_ns)) {
                                fail();
                                ok = false;
                                break;
                            }
                            const uint32_t fb = bar(S::Q_FULL + x);
                            misc->q_loads = 2 * k + x + 1;
                            if (x == 1 && u.nB == 0) {
                                ptx::mbar_arrive(fb);
                                continue;
                            }
                            ptx::mbar_arrive_expect_tx(fb, S::Q_TILE);
                            const int tok = u.first + u.tok0 + x * (kRows / a.G);
#pragma unroll
                            for (int h = 0; h < S::DH; ++h)
                                ptx::tma_load_3d_keep(
                                    sb + S::OFF_Q + x * S::Q_TILE + h * S::Q_ATOM, &tm_q, h * 64,
                                    u.hk * a.G, tok, fb);
                        }
                    }
                    ok = __shfl_sync(kFull, ok, 0);
                    return ok;
                };
                const int q_at = min(n2, S::NS - 2);
                if (!load(0, q_at) || !queries() || !load(q_at, min(n2, S::NS)) ||
                    !wait(S::ANSWER, k)) {
                    // an answer in flight lands before the CTA exits
                    (void)ptx::mbar_wait(bar(S::ANSWER), k & 1, ptx::kDrainLimitNs);
                    break;
                }
                int index;
                Unit nxt;
                nxt.rb = -1;
                if (ptx::cancelled(misc->answer.x, misc->answer.y, index))
                    nxt = find_unit(a, lane, index);
                const uint32_t m = k + 1;
                if (m >= 2 && !wait(S::UNIT_EMPTY + (m & 1), (m >> 1) - 1)) break;
                __syncwarp();
                if (lane == 0) {
                    misc->unit[m & 1] = nxt;
                    ptx::mbar_arrive(bar(S::UNIT_FULL + (m & 1)));
                }
                __syncwarp();
                if (nxt.rb >= 0) {
                    // its queries on their way to L2
                    const int rows = min(kUnit, nxt.len * a.G - nxt.rb * kUnit);
                    for (int r = lane; r < rows; r += 32) {
                        const int t = by_group(a, nxt.rem0 + r);
                        const int h = nxt.rem0 + r - t * a.G;
                        const uint16_t* p =
                            a.q + static_cast<long long>(nxt.first + nxt.tok0 + t) * a.q_ts +
                            static_cast<long long>(nxt.hk * a.G + h) * a.q_hs;
                        ptx::prefetch_l2(p);
                        if (D == 128) ptx::prefetch_l2(p + 64);
                    }
                }
                if (!load(min(n2, S::NS), n2)) break;
                u = nxt;
            }
            // Copies in flight land before the CTA exits, whoever has given up.
            if (lane == 0) {
                for (uint32_t i = t > S::NS ? t - S::NS : 0; i < t; ++i)
                    (void)ptx::mbar_wait(bar(S::FULL + i % S::NS), (i / S::NS) & 1,
                                         ptx::kDrainLimitNs);
                const uint32_t nq = misc->q_loads;
                for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq; ++i)
                    (void)ptx::mbar_wait(bar(S::Q_FULL + (i & 1)), (i >> 1) & 1,
                                         ptx::kDrainLimitNs);
            }
            __syncwarp();
        } else if (warp == kWarpMma) {
            // ================= MMA issuer (the whole warp walks, one lane issues)
            const bool lead = ptx::elect_one();
            const uint32_t id_s = idesc_bf16_f32(kRows, kKeys, false, false);
            const uint32_t id_o = idesc_bf16_f32(kRows, D, false, true);
            auto slot_full = [&](uint32_t t) -> bool {
                return wait(S::FULL + t % S::NS, t / S::NS);
            };
            auto scores = [&](int x, uint32_t t) {  // S_x = Q_x K^T, K in tile t
                const uint32_t kst = sb + S::OFF_RING + (t % S::NS) * S::TILE;
                if (lead) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t ad =
                            smem_desc_sw128(sb + S::OFF_Q + x * S::Q_TILE +
                                                (k >> 2) * S::Q_ATOM + (k & 3) * 32,
                                            16, 1024);
                        const uint64_t bd =
                            smem_desc_sw128(kst + (k >> 2) * S::ATOM + (k & 3) * 32, 16, 1024);
                        ptx::mma_bf16(tmem + S::TM_S + x * kKeys, ad, bd, id_s, k > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit(bar(S::S_FULL + x));
                }
                __syncwarp();
            };
            // O_x += P_x V (or O_x = P_x V), V in tile t, the first keys or the rest
            auto values = [&](int x, uint32_t t, int half, bool add) {
                const uint32_t vst = sb + S::OFF_RING + (t % S::NS) * S::TILE;
                if (lead) {
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k) {
                        if ((k >= kFirstKeys / 16) != (half > 0)) continue;
                        ptx::mma_bf16_ts(tmem + S::TM_O + x * D,
                                         tmem + S::TM_S + x * kKeys + k * 8,
                                         smem_desc_sw128(vst + k * 16 * 128, S::ATOM, 1024), id_o,
                                         (add || k > 0) ? 1u : 0u);
                    }
                }
                __syncwarp();
            };
            auto done = [&](int i) {
                if (lead) ptx::mma_commit(bar(i));
                __syncwarp();
            };
            // The tensor cores' queue is short, and each question asked while it runs dry
            // costs them time: a tile's questions are asked at once, and those that
            // have a "no" for an answer are waited for one by one.
            auto test = [&](int i, uint32_t parity) -> bool {
                return ptx::mbar_test(bar(i), parity & 1);
            };
            uint32_t base = 0, cA = 0, cB = 0, ce = 0;  // tiles, blocks of A and B, edge blocks
            Unit u;
            bool ok = true;
#pragma unroll 1
            for (uint32_t k = 0; ok && next_unit(k, u); ++k) {
                const Span s = span_of(u);
                ok = false;
                if (!slot_full(base) || !wait(S::Q_FULL, k)) break;
                ptx::tc_fence_after();
                scores(0, base);
                if (!wait(S::Q_FULL + 1, k)) break;
                ptx::tc_fence_after();
                if (s.nB > 0) scores(1, base);
                if (s.nA == 1) done(S::Q_FREE);
                if (s.nB <= 1) done(S::Q_FREE + 1);
                done(S::EMPTY + base % S::NS);
                int j = 0;
#pragma unroll 1
                for (; j < s.n; ++j) {
                    const uint32_t tv = base + 2 * j + 1, tk = tv + 1;
                    const int fv = S::FULL + tv % S::NS, fk = S::FULL + tk % S::NS;
                    const uint32_t pv = tv / S::NS, pk = tk / S::NS;
                    if (j >= s.edge) {
                        if (!wait(fv, pv)) break;
                        if (lead) ptx::mbar_arrive(bar(S::ASK));
                        __syncwarp();
                    }
                    auto cleaned = [&]() -> bool {
                        return j < s.edge || wait(S::CLEAN, ce + (j - s.edge));
                    };
                    if (j < s.nA) {
                        const bool last = j + 1 >= s.nA;
                        const bool v = test(fv, pv), h = test(S::P_HALF, cA + j);
                        const bool f = test(S::P_FULL, cA + j), n = last || test(fk, pk);
                        const bool first = __all_sync(kFull, v && h);
                        const bool rest = __all_sync(kFull, f && n);
                        if (!first && !(wait(fv, pv) && wait(S::P_HALF, cA + j))) break;
                        if (!cleaned()) break;
                        ptx::tc_fence_after();
                        values(0, tv, 0, j > 0);
                        if (!rest) {
                            if (!wait(S::P_FULL, cA + j) || !(last || wait(fk, pk))) break;
                            ptx::tc_fence_after();
                        }
                        values(0, tv, 1, true);
                        if (last) {
                            done(S::O_FULL);
                        } else {
                            scores(0, tk);
                            if (j + 2 == s.nA) done(S::Q_FREE);
                        }
                    }
                    if (j < s.nB) {
                        const bool h = test(S::P_HALF + 1, cB + j);
                        const bool f = test(S::P_FULL + 1, cB + j);
                        const bool first = __all_sync(kFull, h);
                        const bool rest = __all_sync(kFull, f);
                        if (!first && !wait(S::P_HALF + 1, cB + j)) break;
                        if (j >= s.nA && (!wait(fv, pv) || !cleaned())) break;
                        ptx::tc_fence_after();
                        values(1, tv, 0, j > 0);
                        if (!rest) {
                            if (!wait(S::P_FULL + 1, cB + j)) break;
                            ptx::tc_fence_after();
                        }
                        values(1, tv, 1, true);
                    }
                    if (j < s.nB) {
                        if (j + 1 >= s.nB) {
                            done(S::O_FULL + 1);
                        } else {
                            if (j + 1 >= s.nA && !wait(fk, pk)) break;
                            scores(1, tk);
                            if (j + 2 == s.nB) done(S::Q_FREE + 1);
                        }
                    }
                    done(S::EMPTY + tv % S::NS);
                    if (j + 1 < s.n) done(S::EMPTY + tk % S::NS);
                }
                if (j < s.n) break;
                ok = true;
                base += 2 * s.n;
                cA += s.nA;
                cB += s.nB;
                ce += max(0, s.n - s.edge);
            }
            done(S::DRAIN);
            (void)ptx::mbar_wait(bar(S::DRAIN), 0, ptx::kDrainLimitNs);
        } else {
            // ================= V tiles of edge blocks: values that are not finite
            // become 0 and are noted.  A warp takes half of the columns.
            constexpr int CPL = D / 16;  // 16-byte chunks of a row taken here
            const int part = warp - kWarpClean;
            const int chunk = part * CPL + lane % CPL;
            uint32_t base = 0, ce = 0;
            Unit u;
            bool ok = true;
#pragma unroll 1
            for (uint32_t k = 0; ok && next_unit(k, u); ++k) {
                const Span s = span_of(u);
                volatile int* dirty = &misc->dirty[k & 3][part];
                if (lane == 0) *dirty = 0;
                __syncwarp();
#pragma unroll 1
                for (int j = s.edge; j < s.n; ++j, ++ce) {
                    // The MMA warp has seen the tile land when it asks; the second
                    // wait makes the copy visible here.
                    const uint32_t t = base + 2 * j + 1;
                    if (!wait(S::ASK, ce) || !wait(S::FULL + t % S::NS, t / S::NS)) {
                        ok = false;
                        break;
                    }
                    uint8_t* tile = smem + S::OFF_RING + (t % S::NS) * S::TILE +
                                    (chunk >> 3) * S::ATOM;
                    auto at = [&](int key) -> uint8_t* {
                        return tile + key * 128 + (((chunk & 7) ^ (key & 7)) << 4);
                    };
                    // x * 0 is NaN for just the values looked for.
                    __nv_bfloat162 sum[4];
                    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = zero;
#pragma unroll 8
                    for (int key = lane / CPL; key < kKeys; key += 32 / CPL) {
                        const uint4 v = *reinterpret_cast<const uint4*>(at(key));
                        const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[i] = __hfma2(w[i], zero, sum[i]);
                    }
                    const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]),
                                                       __hadd2(sum[2], sum[3]));
                    if (__hisnan(__low2bfloat16(all)) || __hisnan(__high2bfloat16(all))) {
                        for (int key = lane / CPL; key < kKeys; key += 32 / CPL) {
                            uint16_t* e = reinterpret_cast<uint16_t*>(at(key));
                            for (int i = 0; i < 8; ++i)
                                if ((e[i] & 0x7f80u) == 0x7f80u) e[i] = 0;
                        }
                        *dirty = 1;
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(S::CLEAN));
                }
                base += 2 * s.n;
            }
        }
    } else {
        // ================= softmax and epilogue: warpgroup x takes tile x
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::SOFT_REGS));
        const int x = warp >> 2;
        const int r = threadIdx.x & 127;  // row of the tile, TMEM lane
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t ts = lanes + S::TM_S + x * kKeys;
        const uint32_t to = lanes + S::TM_O + x * D;
        const uint64_t sc2 = ptx::f2_pack(a.scale_log2, a.scale_log2);
        struct Row {  // this thread's row of a unit
            int nx, edge_x, tok, head, first, edge, hk;
            bool ok;
        };
        auto row_of = [&](const Unit& u) -> Row {
            Row w;
            w.nx = x == 0 ? u.nA : u.nB;
            w.edge = (u.tok0 + 1) / kKeys;
            const int rem = u.rem0 + x * kRows;
            // first block to mask
            w.edge_x = (u.tok0 + by_group(a, rem) + 1) / kKeys;
            w.ok = u.rb * kUnit + x * kRows + r < u.len * a.G;
            const int t = by_group(a, rem + r);
            w.tok = w.ok ? u.tok0 + t : 0;
            w.head = u.hk * a.G + (w.ok ? rem + r - t * a.G : 0);
            w.first = u.first;
            w.hk = u.hk;
            return w;
        };
        // Queries of a unit into the K-major tile, this warp's 32 rows; every
        // score product of the unit before has completed.
        auto load_q = [&](const Row& w) {
            if (a.q_tiles) return;
            if (w.nx > 0) {
                constexpr int LPR = D / 8;  // lanes that move a row, 16 bytes each
                uint8_t* qs = smem + S::OFF_Q + x * S::Q_TILE;
                const long long at =
                    static_cast<long long>(w.first + w.tok) * a.q_ts + w.head * a.q_hs;
                const int c = lane % LPR;
                uint4 v[LPR];
#pragma unroll
                for (int i = 0; i < LPR; ++i) {
                    const int rr = i * (32 / LPR) + lane / LPR;  // row of the warp
                    const long long src = __shfl_sync(kFull, at, rr);
                    v[i] = __ldg(reinterpret_cast<const uint4*>(a.q + src) + c);
                }
#pragma unroll
                for (int i = 0; i < LPR; ++i) {
                    const int rr = (warp & 3) * 32 + i * (32 / LPR) + lane / LPR;
                    // (rows past the sequence hold its first query: never stored)
                    v[i].x = (v[i].x ^ a.q_sign) & a.q_keep;
                    v[i].y = (v[i].y ^ a.q_sign) & a.q_keep;
                    v[i].z = (v[i].z ^ a.q_sign) & a.q_keep;
                    v[i].w = (v[i].w ^ a.q_sign) & a.q_keep;
                    *reinterpret_cast<uint4*>(qs + (c >> 3) * S::Q_ATOM +
                                              sw128_offset(rr, c & 7)) = v[i];
                }
                ptx::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(S::Q_FULL + x));
        };
        uint32_t blocks = 0, ends = 0;  // blocks and units of this tile so far
        Unit u;
        bool have = next_unit(0, u);
        Row w = {};
        if (have) {
            w = row_of(u);
            load_q(w);
        }
#pragma unroll 1
        for (uint32_t k = 0; have; ++k) {
            const bool warp_any = __any_sync(kFull, w.ok);
            float m_ref = kNegInf, l_sum = 0.f;
            bool ok = true;
#pragma unroll 1
            for (int j = 0; j < w.nx; ++j) {
                if (!wait(S::S_FULL + x, blocks + j)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                float s[kKeys];
                if (warp_any) {
                    ptx::tmem_ld32(ts, s);
                    ptx::tmem_ld32(ts + 32, s + 32);
                    ptx::tmem_wait_ld();
                    ptx::tmem_ld32(ts + 64, s + 64);
                    ptx::tmem_ld32(ts + 96, s + 96);
                    const int lim = j >= w.edge_x ? w.tok - j * kKeys : kKeys;  // last key seen
                    float mp[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mp[i] = kNegInf;
                    // the first half's maxima while the second half is on its way
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1) ptx::tmem_wait_ld();
                        if (j >= w.edge_x) {
#pragma unroll
                            for (int i = 64 * h; i < 64 * h + 64; ++i)
                                if (i > lim) s[i] = kNegInf;
                        }
#pragma unroll
                        for (int i = 64 * h; i < 64 * h + 64; i += 2)
                            mp[(i >> 1) & 7] = ptx::fmax3(mp[(i >> 1) & 7], s[i], s[i + 1]);
                    }
                    const float mx = ptx::fmax3(ptx::fmax3(mp[0], mp[1], mp[2]),
                                                ptx::fmax3(mp[3], mp[4], mp[5]),
                                                fmaxf(mp[6], mp[7])) *
                                     a.scale_log2;
                    float alpha = 1.f;
                    bool rescale = false;
                    if (j == 0) {
                        m_ref = mx;
                    } else if (mx > m_ref + 8.f) {
                        alpha = ptx::ex2(m_ref - mx);
                        m_ref = mx;
                        l_sum *= alpha;
                        rescale = true;
                    }
                    // S_x(j) was issued behind O_x += P V of block j - 1 and has
                    // completed, so O is at rest until this block's P is handed over.
                    if (__any_sync(kFull, rescale)) {
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            ptx::tmem_ld32(to + c, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= alpha;
                            ptx::tmem_st32(to + c, o);
                        }
                    }
                    const float neg_m = m_ref == kNegInf ? 0.f : -m_ref;
                    const uint64_t nm2 = ptx::f2_pack(neg_m, neg_m);
#pragma unroll
                    for (int c = 0; c < kKeys; c += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = c; i < c + 32; i += 2) {
                            float e0, e1;
                            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(s[i], s[i + 1]), sc2, nm2), e0,
                                           e1);
                            s[i] = ptx::ex2(e0);
                            s[i + 1] = ptx::ex2(e1);
                            pk[(i - c) / 2] = pack_bf16(s[i], s[i + 1]);
                        }
                        ptx::tmem_st16(ts + c / 2, pk);
                        if (c + 32 == kFirstKeys) {
                            // the tensor cores may start on these keys
                            ptx::tmem_wait_st();
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(bar(S::P_HALF + x));
                        }
                    }
                    ptx::tmem_wait_st();
                } else if (lane == 0) {
                    ptx::mbar_arrive(bar(S::P_HALF + x));
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(S::P_FULL + x));
                if (warp_any) {  // the row's sum, off the tensor cores' path
                    uint64_t sp2[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sp2[i] = ptx::f2_pack(s[2 * i], s[2 * i + 1]);
#pragma unroll
                    for (int i = 8; i < kKeys; i += 2)
                        sp2[(i >> 1) & 3] =
                            ptx::f2_add(sp2[(i >> 1) & 3], ptx::f2_pack(s[i], s[i + 1]));
                    float p[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) ptx::f2_unpack(sp2[i], p[2 * i], p[2 * i + 1]);
                    l_sum += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
                }
            }
            if (!ok) break;
            blocks += w.nx;
            // ---- the next unit's queries, so that its first scores are made beside
            // this epilogue
            const Row end = w;
            have = next_unit(k + 1, u);
            if (have) {
                w = row_of(u);
                load_q(w);
            }
            // ---- epilogue
            if (end.nx == 0) continue;
            if (!wait(S::O_FULL + x, ends)) break;
            ++ends;
            ptx::tc_fence_after();
            if (!warp_any) continue;
            const float inv = 1.f / l_sum;
            uint8_t* stg = smem + S::OFF_OUT + warp * (32 * 128);
            const volatile int* d3 = misc->dirty[k & 3];
            const bool dirty = (d3[0] | d3[1]) != 0;
            const long long row =
                static_cast<long long>(end.first + end.tok) * a.Hq + end.head;
            // where the row goes, from the warp's first row on (which exists); -1: nowhere
            const long long row_0 = __shfl_sync(kFull, row, 0);
            const int rel = end.ok ? static_cast<int>(row - row_0) : -1;
            const bool box = a.o_tiles && !dirty && __all_sync(kFull, end.ok);
            // 64 columns at a time through this warp's staging rows, so that a store
            // instruction covers whole 128-byte pieces of four rows.
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
                float o[64];
                ptx::tmem_ld32(to + c, o);
                ptx::tmem_ld32(to + c + 32, o + 32);
                ptx::tmem_wait_ld();
                if (lane == 0) ptx::bulk_wait_read();  // the staging rows' last box
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        pk[e] = pack_bf16(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv);
                    *reinterpret_cast<uint4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                        make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                if (box) {
                    // (32 rows are whole tokens, and the first row's head is the group's)
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        ptx::tma_store_3d(&tm_o, c, end.head, end.first + end.tok,
                                          sb + S::OFF_OUT + warp * (32 * 128));
                    continue;
                }
                __syncwarp();
                const int ch = lane & 7;
                uint16_t* dst = a.out + row_0 * D + c + ch * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = 4 * i + (lane >> 3);
                    const int to_row = __shfl_sync(kFull, rel, rr);
                    const uint4 v = *reinterpret_cast<const uint4*>(
                        stg + rr * 128 + ((ch ^ (rr & 7)) << 4));
                    if (to_row >= 0)
                        *reinterpret_cast<uint4*>(dst + static_cast<long long>(to_row) * D) = v;
                }
                __syncwarp();
            }
            if (dirty && end.ok) {
                // (rare) what was cleared, for the rows that see it: a probability
                // times NaN or an infinity is that again, whatever it is added to
#pragma unroll 1
                for (int c = 0; c < D; ++c) {
                    float odd = 0.f;
#pragma unroll 1
                    for (int key = end.edge * kKeys; key <= end.tok; ++key) {
                        const uint32_t b = __ldg(
                            a.v + static_cast<long long>(end.first + key) * a.v_ts +
                            end.hk * a.v_hs + c);
                        if ((b & 0x7f80u) == 0x7f80u) odd += __uint_as_float(b << 16);
                    }
                    uint16_t* at = a.out + row * D + c;
                    if (odd != 0.f)
                        *at = static_cast<uint16_t>(pack_bf16(
                            __uint_as_float(static_cast<uint32_t>(*at) << 16) + odd, 0.f));
                }
            }
            if (end.ok) a.lse[row] = (m_ref + log2f(l_sum)) * kLn2;
            ptx::tc_fence_before();
        }
        if (lane == 0) ptx::bulk_wait();
    }

    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// [N][H][d] rows in boxes of 128 tokens x one head x 64 columns; a head stride of
// 0 (one head standing for all) becomes an extent of 1.
bool encode_rows(CUtensorMap* map, const void* base, int N, int H, int d, long long ts,
                 long long hs) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d),
                                hs != 0 ? static_cast<cuuint64_t>(H) : 1,
                                static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[2] = {hs != 0 ? static_cast<cuuint64_t>(hs) * 2 : 16,
                                   N > 1 ? static_cast<cuuint64_t>(ts) * 2 : 16};
    const cuuint32_t box[3] = {64, 1, kKeys};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

// The same rows in boxes of `tokens` tokens x G heads x 64 columns, in which a
// row is token * G + head.
bool encode_groups(CUtensorMap* map, const void* base, int N, int H, int d, long long ts,
                   long long hs, int G, int tokens) {
    if ((N > 1 && ts == 0) || (H > 1 && hs == 0)) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                                static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[2] = {H > 1 ? static_cast<cuuint64_t>(hs) * 2 : 16,
                                   N > 1 ? static_cast<cuuint64_t>(ts) * 2 : 16};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tokens)};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D>
cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                           const CUtensorMap& tq, const CUtensorMap& to, long long ctas,
                           cudaStream_t stream) {
    static std::atomic<unsigned long long> configured{0};  // by device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if ((configured.load() & bit) == 0) {
        e = cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape<D>::SMEM);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return launch_dependent(prefill_kernel<D>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads),
                            Shape<D>::SMEM, stream, tk, tv, tq, to, a);
}

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" int tree_attn_prefill(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                 long long q_token_stride, long long q_head_stride,
                                 long long k_token_stride, long long k_head_stride,
                                 long long v_token_stride, long long v_head_stride,
                                 const int32_t* cu_seqlens, uint16_t* out, float* lse, int B,
                                 int N, int Hq, int Hkv, int d, float softmax_scale,
                                 int32_t* status, void* stream) {
    if (B < 0 || N < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > 65535 ||
        (d != 64 && d != 128) || !std::isfinite(softmax_scale) || q_token_stride < 0 ||
        q_head_stride < 0 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 ||
        v_head_stride < 0 || (N > 1 && (k_token_stride == 0 || v_token_stride == 0)) ||
        static_cast<long long>(N) * (Hq / Hkv) >= (1LL << 31) - kUnit)
        return TREE_ATTN_ERR_SHAPE;
    // One CTA per 256 rows of a sequence and KV head; the lengths are on the
    // device, so the grid is the largest it can be and the rest end at once.
    const long long ctas =
        (static_cast<long long>(N) * (Hq / Hkv) / kUnit + B) * static_cast<long long>(Hkv);
    if (ctas > 0x7fffffffLL) return TREE_ATTN_ERR_SHAPE;
    if (B == 0 || N == 0) return TREE_ATTN_OK;
    if (!q || !k || !v || !cu_seqlens || !out || !lse) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(q, 16) || !ptr_aligned(k, 16) || !ptr_aligned(v, 16) ||
        !ptr_aligned(out, 16) || !ptr_aligned(lse, 4) || !ptr_aligned(cu_seqlens, 4) ||
        !ptr_aligned(status, 4) || q_token_stride % 8 != 0 || q_head_stride % 8 != 0 ||
        k_token_stride % 8 != 0 || k_head_stride % 8 != 0 || v_token_stride % 8 != 0 ||
        v_head_stride % 8 != 0)
        return TREE_ATTN_ERR_ALIGN;
    CUtensorMap tk, tv;
    if (!encode_rows(&tk, k, N, Hkv, d, k_token_stride, k_head_stride) ||
        !encode_rows(&tv, v, N, Hkv, d, v_token_stride, v_head_stride))
        return TREE_ATTN_ERR_CUDA;
    PrefillArgs a;
    a.q = q;
    a.v = v;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.k_heads = k_head_stride != 0;
    a.v_heads = v_head_stride != 0;
    a.cu = cu_seqlens;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.inv_g = 1.f / static_cast<float>(a.G);
    // The kernel looks for the largest raw score, so a negative scale turns the
    // queries round instead, and a scale of zero clears them.
    a.q_sign = softmax_scale < 0.f ? 0x80008000u : 0u;
    a.q_keep = softmax_scale == 0.f ? 0u : 0xffffffffu;
    a.scale_log2 = softmax_scale == 0.f
                       ? 1.f
                       : static_cast<float>(std::fabs(static_cast<double>(softmax_scale)) *
                                            1.4426950408889634);
    a.wait_ns = wait_limit_ns();
    // Queries and results move as whole boxes where a warp's 32 rows are whole
    // tokens and the queries go in as they are (16 sequences of up to 2048 tokens, 8
    // heads to a KV head: 377 us); else row by row through registers (405 us).
    CUtensorMap tq = tk, to = tk;
    const bool whole = 32 % a.G == 0;
    a.q_tiles = whole && softmax_scale > 0.f &&
                encode_groups(&tq, q, N, Hq, d, q_token_stride, q_head_stride, a.G, kRows / a.G);
    a.o_tiles = whole && encode_groups(&to, out, N, Hq, d, static_cast<long long>(Hq) * d, d, a.G,
                                       32 / a.G);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d == 128 ? launch_prefill<128>(a, tk, tv, tq, to, ctas, st)
                                   : launch_prefill<64>(a, tk, tv, tq, to, ctas, st);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
