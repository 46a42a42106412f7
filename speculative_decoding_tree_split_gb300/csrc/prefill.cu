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
// * Keys a row may not see get a score of -inf by index, whatever K holds.
//   V of such keys still meets P = 0 in the tensor cores, and 0 * NaN is not 0:
//   in blocks that some row does not see whole, two warps clear the non-finite
//   values of the V tile and note where they stood; the epilogue puts them back
//   into the rows that see them.
// * Units are taken longest first (the grid is one CTA per unit).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/tree_attn.h"
#include "kernels.cuh"
#include "launch.cuh"
#include "layout.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kKeys = 128;           // keys of a block
constexpr int kUnit = 2 * kRows;     // rows of a unit
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpClean = 10;
constexpr int kThreads = 384;        // two softmax warpgroups and one of helpers
// Registers: 168 a thread at launch; the helpers give theirs to the softmax,
// which holds a row's 128 scores.  256 * 208 + 128 * 56 <= 384 * 168.
constexpr int kSoftRegs = 208, kHelpRegs = 56;

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

struct PrefillArgs {
    const uint16_t* q;
    long long q_ts, q_hs;  // token and head strides (elements)
    int k_heads, v_heads;  // 0: one head stands for all (stride 0)
    const int32_t* cu;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int B, N, Hq, Hkv, G;
    float scale_log2;      // >= 0
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
    static constexpr int NS = D == 128 ? 5 : 8;    // ring slots, K and V in turn
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + 2 * Q_TILE;
    static constexpr int OFF_FIRST = OFF_RING + NS * TILE;  // int [3][D]: see clean()
    static constexpr int OFF_MISC = OFF_FIRST + 3 * D * 4;
    static constexpr int OFF_BAR = OFF_MISC + 64;
    static constexpr int FULL = 0;
    static constexpr int EMPTY = NS;
    static constexpr int S_FULL = 2 * NS;      // [2] by tile
    static constexpr int P_FULL = S_FULL + 2;  // [2]: all of P
    static constexpr int O_FULL = S_FULL + 4;  // [2]
    static constexpr int Q_FULL = S_FULL + 6;  // [2]
    static constexpr int ASK = S_FULL + 8;    // V of an edge block has landed: clean it
    static constexpr int CLEAN = S_FULL + 9;  // it is clean
    static constexpr int P_HALF = S_FULL + 10;  // [2]: P of the first 64 keys
    static constexpr int DRAIN = S_FULL + 12;
    static constexpr int NBAR = S_FULL + 13;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 1024;  // + alignment slack
    // TMEM: S of both tiles (P over them), then O of both.
    static constexpr int TM_S = 0;
    static constexpr int TM_O = 2 * kKeys;
    static_assert(TM_O + 2 * D <= 512, "TMEM budget");
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
    static_assert(SMEM > 114 * 1024, "one CTA per SM keeps TMEM allocation uncontended");
};

struct Misc {
    uint32_t tmem_base;
    int abort;
    int dirty;  // clean() found something
};

struct Unit {
    int b, hk, rb;
    int first, len;  // packed rows of the sequence
};

// Row blocks of sequence b (0 where its range is out of order or empty).
__device__ __forceinline__ int row_blocks(const PrefillArgs& a, int b) {
    if (b >= a.B) return 0;
    const int lo = a.cu[b], hi = a.cu[b + 1];
    if (lo < 0 || hi < lo || hi > a.N) return 0;
    const long long rows = static_cast<long long>(hi - lo) * a.G;
    return static_cast<int>((rows + kUnit - 1) / kUnit);
}

// Unit blockIdx.x in the order of falling row-block index (so of falling work),
// KV heads innermost; false past the last.  One warp, every lane gets it.  With
// n_b row blocks in sequence b, the units of index >= r number
// sum_b max(0, n_b - r), so the index of unit u is found by halving.
__device__ bool find_unit(const PrefillArgs& a, int lane, Unit& u) {
    const int id = static_cast<int>(blockIdx.x) / a.Hkv;
    u.hk = static_cast<int>(blockIdx.x) % a.Hkv;
    const int n0 = row_blocks(a, lane);  // the first 32 sequences stay here
    auto count = [&](int r) -> int {
        int n = max(0, n0 - r);
        for (int b = 32; b < a.B; b += 32) n += max(0, row_blocks(a, b + lane) - r);
        return __reduce_add_sync(kFull, n);
    };
    if (id >= count(0)) return false;
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
            u.b = b + at;
            u.first = a.cu[u.b];
            u.len = a.cu[u.b + 1] - u.first;
            return true;
        }
        rest -= c;
    }
    return false;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a) {
    using S = Shape<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sb = raw_addr + pad;
    Misc* misc = reinterpret_cast<Misc*>(smem + S::OFF_MISC);
    volatile int* abort_flag = &misc->abort;
    int* first_bad = reinterpret_cast<int*>(smem + S::OFF_FIRST);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sb + S::OFF_BAR + 8u * i; };

    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += kThreads)
            if (a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.N)
                report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    Unit u;
    if (!find_unit(a, lane, u)) return;  // the same in every warp

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
            ptx::mbar_init(bar(S::Q_FULL + i), 4);
        }
        ptx::mbar_init(bar(S::ASK), 1);
        ptx::mbar_init(bar(S::CLEAN), 2);
        ptx::mbar_init(bar(S::DRAIN), 1);
        misc->abort = 0;
        misc->dirty = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(ptx::smem_u32(&misc->tmem_base), 512);
        ptx::tmem_relinquish();
    }
    for (int i = threadIdx.x; i < 3 * D; i += kThreads) first_bad[i] = INT_MAX;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc->tmem_base;
    auto fail = [&]() {
        *abort_flag = 1;
        report(a.status, TREE_ATTN_STATUS_TIMEOUT);
    };

    // Rows of the unit: row r of the sequence is token r / G, head r % G of the
    // group.  Tile x holds rows [row0 + 128 x, ...); its keys end with its last
    // row's token.
    const int rows = u.len * a.G;  // fits: N * G < 2^31 (checked on the host)
    const int row0 = u.rb * kUnit;
    auto blocks_of = [&](int x) -> int {
        const int lo = row0 + x * kRows;
        if (lo >= rows) return 0;
        return (min(lo + kRows, rows) - 1) / a.G / kKeys + 1;
    };
    const int nA = blocks_of(0), nB = blocks_of(1);
    const int n = max(nA, nB);
    // Blocks from this one on hold keys that some row of the unit does not see.
    const int edge = (row0 / a.G + 1) / kKeys;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kHelpRegs));
        if (warp == kWarpTma) {
            // ================= copies (one lane): K0, V0, K1, V1, ...
            if (lane == 0) {
                bool ok = true;
                int t = 0;
                const int hk_k = a.k_heads ? u.hk : 0, hk_v = a.v_heads ? u.hk : 0;
#pragma unroll 1
                for (; t < 2 * n; ++t) {
                    const int s = t % S::NS;
                    if (t >= S::NS &&
                        !ptx::mbar_wait(bar(S::EMPTY + s), (t / S::NS - 1) & 1, a.wait_ns)) {
                        fail();
                        ok = false;
                        break;
                    }
                    if (*abort_flag) {
                        ok = false;
                        break;
                    }
                    const bool is_v = t & 1;
                    const int tok = u.first + (t >> 1) * kKeys;
                    const int y = is_v ? hk_v : hk_k;
                    const uint32_t dst = sb + S::OFF_RING + s * S::TILE;
                    ptx::mbar_arrive_expect_tx(bar(S::FULL + s), S::TILE);
#pragma unroll
                    for (int h = 0; h < S::DH; ++h)
                        ptx::tma_load_3d_keep(dst + h * S::ATOM, is_v ? &tm_v : &tm_k, h * 64, y,
                                              tok, bar(S::FULL + s));
                }
                if (!ok) {
                    for (int k = t > S::NS ? t - S::NS : 0; k < t; ++k)
                        (void)ptx::mbar_wait(bar(S::FULL + k % S::NS), (k / S::NS) & 1,
                                             ptx::kDrainLimitNs);
                }
            }
        } else if (warp == kWarpMma) {
            // ================= MMA issuer (the whole warp walks, one lane issues)
            const bool lead = ptx::elect_one();
            const uint32_t id_s = idesc_bf16_f32(kRows, kKeys, false, false);
            const uint32_t id_o = idesc_bf16_f32(kRows, D, false, true);
            bool ok = true;
            auto wait = [&](int i, int parity) -> bool {
                const bool all =
                    __all_sync(kFull, ptx::mbar_wait(bar(i), parity, a.wait_ns));
                if (!all) fail();
                return all;
            };
            auto slot_full = [&](int t) -> bool {
                return wait(S::FULL + t % S::NS, (t / S::NS) & 1);
            };
            auto scores = [&](int x, int j) {  // S_x = Q_x K_j^T
                const uint32_t kst = sb + S::OFF_RING + (2 * j % S::NS) * S::TILE;
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
            auto values = [&](int x, int j, int half) {  // O_x += P_x V_j, 64 keys
                const uint32_t vst = sb + S::OFF_RING + ((2 * j + 1) % S::NS) * S::TILE;
                if (lead) {
#pragma unroll
                    for (int i = 0; i < kKeys / 32; ++i) {
                        const int k = half * (kKeys / 32) + i;
                        ptx::mma_bf16_ts(tmem + S::TM_O + x * D,
                                         tmem + S::TM_S + x * kKeys + k * 8,
                                         smem_desc_sw128(vst + k * 16 * 128, S::ATOM, 1024), id_o,
                                         (j > 0 || k > 0) ? 1u : 0u);
                    }
                }
                __syncwarp();
            };
            auto done = [&](int i) {
                if (lead) ptx::mma_commit(bar(i));
                __syncwarp();
            };
            auto cleaned = [&](int j) -> bool {
                return j < edge || wait(S::CLEAN, (j - edge) & 1);
            };
            ok = slot_full(0) && wait(S::Q_FULL, 0);
            if (ok) {
                ptx::tc_fence_after();
                scores(0, 0);
                if (nB > 0) {
                    ok = wait(S::Q_FULL + 1, 0);
                    if (ok) {
                        ptx::tc_fence_after();
                        scores(1, 0);
                    }
                }
                done(S::EMPTY + 0);
            }
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) {
                if (!slot_full(2 * j + 1)) break;
                if (j >= edge) {
                    if (lead) ptx::mbar_arrive(bar(S::ASK));
                    __syncwarp();
                }
                if (j < nA) {
                    if (!wait(S::P_HALF, j & 1) || !cleaned(j)) break;
                    ptx::tc_fence_after();
                    values(0, j, 0);
                    if (!wait(S::P_FULL, j & 1)) break;
                    ptx::tc_fence_after();
                    values(0, j, 1);
                    if (j + 1 >= nA) {
                        done(S::O_FULL);
                    } else {
                        if (!slot_full(2 * j + 2)) break;
                        scores(0, j + 1);
                    }
                }
                if (j < nB) {
                    if (!wait(S::P_HALF + 1, j & 1) || (j >= nA && !cleaned(j))) break;
                    ptx::tc_fence_after();
                    values(1, j, 0);
                    if (!wait(S::P_FULL + 1, j & 1)) break;
                    ptx::tc_fence_after();
                    values(1, j, 1);
                }
                done(S::EMPTY + (2 * j + 1) % S::NS);
                if (j < nB) {
                    if (j + 1 >= nB) {
                        done(S::O_FULL + 1);
                    } else {
                        if (!slot_full(2 * j + 2)) break;
                        scores(1, j + 1);
                    }
                }
                if (j + 1 < n) done(S::EMPTY + (2 * j + 2) % S::NS);
            }
            done(S::DRAIN);
            (void)ptx::mbar_wait(bar(S::DRAIN), 0, ptx::kDrainLimitNs);
        } else {
            // ================= clean(): V tiles of the edge blocks.  For each
            // column the first key that holds NaN, +inf, -inf is noted.
            const int part = warp - kWarpClean;
#pragma unroll 1
            for (int j = edge; j < n; ++j) {
                // The MMA warp has seen the tile land when it asks; the second
                // wait makes the copy visible here.
                const int t = 2 * j + 1;
                if (!__all_sync(kFull,
                                ptx::mbar_wait(bar(S::ASK), (j - edge) & 1, a.wait_ns) &&
                                    ptx::mbar_wait(bar(S::FULL + t % S::NS), (t / S::NS) & 1,
                                                   a.wait_ns))) {
                    fail();
                    break;
                }
                uint8_t* tile = smem + S::OFF_RING + (t % S::NS) * S::TILE;
                // x * 0 is NaN for just the values looked for.
                __nv_bfloat162 sum[4];
                const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] = zero;
#pragma unroll 8
                for (int i = part * 32 + lane; i < S::TILE / 16; i += 64) {
                    const uint4 v = *reinterpret_cast<const uint4*>(tile + i * 16);
                    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) sum[k] = __hfma2(w[k], zero, sum[k]);
                }
                const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]),
                                                   __hadd2(sum[2], sum[3]));
                if (__hisnan(__low2bfloat16(all)) || __hisnan(__high2bfloat16(all))) {
                    for (int i = part * 32 + lane; i < S::TILE / 16; i += 64) {
                        // 16-byte chunk i: atom column, row (key), swizzled chunk
                        const int key = (i % (S::ATOM / 16)) / 8;
                        const int c0 = (i / (S::ATOM / 16)) * 64 + ((i & 7) ^ (key & 7)) * 8;
                        uint16_t* e = reinterpret_cast<uint16_t*>(tile + i * 16);
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t x = e[k];
                            if ((x & 0x7f80u) != 0x7f80u) continue;
                            const int kind = (x & 0x7fu) != 0 ? 0 : ((x >> 15) ? 2 : 1);
                            atomicMin(first_bad + kind * D + c0 + k, j * kKeys + key);
                            e[k] = 0;
                            misc->dirty = 1;
                        }
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(S::CLEAN));
            }
        }
    } else {
        // ================= softmax and epilogue: warpgroup x takes tile x
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int x = warp >> 2;
        const int r = threadIdx.x & 127;  // row of the tile, TMEM lane
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t ts = lanes + S::TM_S + x * kKeys;
        const uint32_t to = lanes + S::TM_O + x * D;
        const int nx = x == 0 ? nA : nB;
        const int row = row0 + x * kRows + r;
        const bool row_ok = row < rows;
        const int tok = row_ok ? row / a.G : 0;
        const int head = u.hk * a.G + (row_ok ? row % a.G : 0);
        constexpr int LPR = D / 8;  // lanes that move a row, 16 bytes each
        // ---- queries into the K-major tile, this warp's 32 rows
        if (nx > 0) {
            uint8_t* qs = smem + S::OFF_Q + x * S::Q_TILE;
            const long long at = static_cast<long long>(u.first + tok) * a.q_ts + head * a.q_hs;
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
                *reinterpret_cast<uint4*>(qs + (c >> 3) * S::Q_ATOM + sw128_offset(rr, c & 7)) =
                    v[i];
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(S::Q_FULL + x));
        }
        auto wait = [&](int i, int parity) -> bool {
            const bool all = __all_sync(kFull, ptx::mbar_wait(bar(i), parity, a.wait_ns));
            if (!all) fail();
            return all;
        };
        const bool warp_any = __any_sync(kFull, row_ok);
        const int edge_x = ((row0 + x * kRows) / a.G + 1) / kKeys;  // first block to mask
        float m_ref = kNegInf, l_sum = 0.f;
        bool ok = true;
        const uint64_t sc2 = ptx::f2_pack(a.scale_log2, a.scale_log2);
#pragma unroll 1
        for (int j = 0; j < nx; ++j) {
            if (!wait(S::S_FULL + x, j & 1)) {
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
                const int lim = j >= edge_x ? tok - j * kKeys : kKeys;  // last key seen
                float mp[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mp[i] = kNegInf;
                // the first half's maxima while the second half is on its way
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1) ptx::tmem_wait_ld();
                    if (j >= edge_x) {
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
                    if (c == 32) {
                        // the tensor cores may start on these 64 keys
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
        // ---- epilogue: rows out through this warp's part of the query tile (all
        // its score products have completed)
        if (ok && nx > 0 && wait(S::O_FULL + x, 0)) {
            ptx::tc_fence_after();
            if (warp_any) {
                const float inv = 1.f / l_sum;
                const bool dirty = *reinterpret_cast<volatile int*>(&misc->dirty) != 0;
                uint8_t* stg = smem + S::OFF_Q + x * S::Q_TILE + (warp & 3) * 32 * D * 2;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    ptx::tmem_ld32(to + c, o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= inv;
                    if (dirty) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const bool nan = first_bad[c + i] <= tok;
                            const bool up = first_bad[D + c + i] <= tok;
                            const bool dn = first_bad[2 * D + c + i] <= tok;
                            if (up) o[i] += __builtin_huge_valf();
                            if (dn) o[i] -= __builtin_huge_valf();
                            if (nan) o[i] = __int_as_float(0x7fffffff);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ch = c / 8 + i;  // 16-byte chunk of the row
                        *reinterpret_cast<uint4*>(stg + lane * (D * 2) +
                                                  ((ch ^ (lane & 7)) << 4)) =
                            make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]),
                                       pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                       pack_bf16(o[8 * i + 4], o[8 * i + 5]),
                                       pack_bf16(o[8 * i + 6], o[8 * i + 7]));
                    }
                }
                if (row_ok)
                    a.lse[static_cast<long long>(u.first + tok) * a.Hq + head] =
                        (m_ref + log2f(l_sum)) * kLn2;
                __syncwarp();
                const long long at =
                    (static_cast<long long>(u.first + tok) * a.Hq + head) * D;
#pragma unroll
                for (int i = 0; i < LPR; ++i) {
                    const int rr = i * (32 / LPR) + lane / LPR;
                    const int ch = lane % LPR;
                    const long long dst = __shfl_sync(kFull, at, rr);
                    if (__shfl_sync(kFull, row_ok, rr))
                        *reinterpret_cast<uint4*>(a.out + dst + ch * 8) =
                            *reinterpret_cast<const uint4*>(stg + rr * (D * 2) +
                                                            ((ch ^ (rr & 7)) << 4));
                }
            }
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

template <int D>
cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                           long long ctas, cudaStream_t stream) {
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
                            Shape<D>::SMEM, stream, tk, tv, a);
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
    // device, so the grid is the largest it can be and the rest return at once.
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
    // The kernel looks for the largest raw score, so a negative scale turns the
    // queries round instead, and a scale of zero clears them.
    a.q_sign = softmax_scale < 0.f ? 0x80008000u : 0u;
    a.q_keep = softmax_scale == 0.f ? 0u : 0xffffffffu;
    a.scale_log2 = softmax_scale == 0.f
                       ? 1.f
                       : static_cast<float>(std::fabs(static_cast<double>(softmax_scale)) *
                                            1.4426950408889634);
    a.wait_ns = wait_limit_ns();
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d == 128 ? launch_prefill<128>(a, tk, tv, ctas, st)
                                   : launch_prefill<64>(a, tk, tv, ctas, st);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
