// pages.cu -- the pages of a paged cache as managed things: copied, forked
// (rows of the next step made from rows of this one: sharing, copy on write,
// growth, release) and compacted.
//
// A page's reference count is the only state: 0 is free, and a page handed out
// is always the lowest free one not yet handed out, in order of (row, slot), so
// that results do not depend on timing.  Counts and tables go from inputs to
// outputs; what this call frees is not handed out by it, so no page is read
// and written by the copies.
//
// A plan is a few KB to a few MB of integers with four dependent phases: one
// cluster of CTAs runs them with hardware barriers in between, in one launch; it is
// bound by their latency (9 to 14 us from cold caches).  The copies, with the new table
// made beside them, are bound by memory traffic (515 MB moved in 77 us, 6.7 TB/s).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/tree_attn.h"
#include "cluster.cuh"
#include "launch.cuh"
#include "layout.h"
#include "ptx.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxCtas = 8;

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

// ---------------------------------------------------------------------------
// What both plans use: prefix sums of one CTA, and runs over the page counts.
// ---------------------------------------------------------------------------

// Exclusive prefix of v over the CTA's threads; the sum in `total`.
template <int WARPS = kPlanWarps>
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const int s = warp_sums[w];
        before += w < warp ? s : 0;
        all += s;
    }
    total = all;
    return before + x - v;
}

// The part [lo, hi) of the pages that a CTA of the cluster looks after.
__device__ __forceinline__ void my_pages(int num_pages, int& lo, int& hi) {
    const long long ctas = ptx::cluster_size(), r = ptx::cluster_rank();
    lo = static_cast<int>(num_pages * r / ctas);
    hi = static_cast<int>(num_pages * (r + 1) / ctas);
}

// ---------------------------------------------------------------------------
// Fork.  Row i continues row p = src[i] with its L = seq_lens[p] tokens (p = -2: a
// new row, L = 0; p = -1: no row, no pages):
//   slots before floor(L / P)   p's pages, shared;
//   slots up to (L + reserve)   p's own page where i is p's first row and no
//                               other reference to that page exists, else a new
//                               page; the one that holds tokens is copied;
//   behind                      none.
// counts' = counts - (entries of the old table) + (entries of the new one).
// ---------------------------------------------------------------------------
struct ForkArgs {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* refs;
    const int32_t* src;
    const int32_t* reserve;  // nullable: reserve_all for every row
    int reserve_all;
    int32_t* table_out;
    int32_t* lens_out;
    int32_t* refs_out;
    int rows_in, rows_out, max_pages, P, num_pages;
    // workspace
    int32_t* copy_src;  // [rows_out]
    int32_t* copy_dst;  // [rows_out]
    int32_t* count;     // [1]
    int32_t* free_all;  // [1] free pages
    int32_t* free_of;   // [kMaxCtas] free pages of each CTA's part
    int32_t* children;  // [rows_in]
    int32_t* eldest;    // [rows_in]
    int32_t* wants;     // [rows_out] new pages, 2^30 added if one is a copy
    int32_t* base;      // [rows_out] new pages of the rows before
    int32_t* copies;    // [rows_out] copies of the rows before
    int32_t* list;      // [num_pages] free pages in order
    int32_t* status;
};

struct Row {
    int parent;  // -1: no row, -2: a new one
    int L, full, need;
    bool eldest;
};

__device__ __forceinline__ bool entry_ok(int e, int num_pages) { return e >= 0 && e < num_pages; }

__device__ __forceinline__ Row row_of(const ForkArgs& a, int i, const int32_t* eldest) {
    Row r;
    r.parent = a.src[i];
    r.L = r.full = r.need = 0;
    r.eldest = false;
    if (r.parent < -2 || r.parent >= a.rows_in) {
        report(a.status, TREE_ATTN_STATUS_BAD_ROW);
        r.parent = -1;
    }
    if (r.parent == -1) return r;
    bool bad = false;
    if (r.parent >= 0) {
        r.L = clamp_seq_len(a.lens[r.parent], a.P, a.max_pages, bad);
        r.eldest = eldest[r.parent] == i;
    }
    if (bad) {
        report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
        r.L = 0;
    }
    const int more = a.reserve != nullptr ? a.reserve[i] : a.reserve_all;
    const long long end = static_cast<long long>(r.L) + max(more, 0);
    const long long need = (end + a.P - 1) / a.P;
    if (need > a.max_pages) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    r.full = r.L / a.P;
    r.need = static_cast<int>(min(need, static_cast<long long>(a.max_pages)));
    return r;
}

// Whether row r keeps its parent's entry e behind the full pages.
__device__ __forceinline__ bool keeps(const ForkArgs& a, const Row& r, int e) {
    return r.eldest && entry_ok(e, a.num_pages) && a.refs[e] == 1;
}

// Rows whose children and eldest child a CTA keeps in shared memory.
constexpr int kHeldRows = 4096;

// The plan: new pages of every row, and which pages are copied.  The table itself is made
// beside the copies (fork_row, fork_release).
__global__ void __launch_bounds__(kPlanThreads) fork_kernel(const ForkArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ int sums[kPlanWarps];
    __shared__ int children[kHeldRows], eldest[kHeldRows];
    const int tid = threadIdx.x, lane = tid & 31;
    const int ctas = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    const int gtid = rank * kPlanThreads + tid, gthreads = ctas * kPlanThreads;
    const int gwarp = gtid >> 5, gwarps = gthreads >> 5;
    int lo, hi;
    my_pages(a.num_pages, lo, hi);

    // Counts carried over, free pages counted; every row's children.  Where rows are not
    // too many, each CTA finds all of them for itself.
    const bool held = a.rows_in <= kHeldRows;
    if (held) {
        for (int p = tid; p < a.rows_in; p += kPlanThreads) {
            children[p] = 0;
            eldest[p] = 0x7fffffff;
        }
        __syncthreads();
        for (int i = tid; i < a.rows_out; i += kPlanThreads) {
            const int p = a.src[i];
            if (p >= 0 && p < a.rows_in) {
                atomicAdd(children + p, 1);
                atomicMin(eldest + p, i);
            }
        }
    } else {
        for (int p = gtid; p < a.rows_in; p += gthreads) {
            a.children[p] = 0;
            a.eldest[p] = 0x7fffffff;
        }
        ptx::cluster_sync();
        for (int i = gtid; i < a.rows_out; i += gthreads) {
            const int p = a.src[i];
            if (p >= 0 && p < a.rows_in) {
                atomicAdd(a.children + p, 1);
                atomicMin(a.eldest + p, i);
            }
        }
        ptx::cluster_sync();
    }
    int mine = 0;
#pragma unroll 4
    for (int p = lo + tid; p < hi; p += kPlanThreads) {
        const int c = a.refs[p];
        a.refs_out[p] = c;
        mine += c == 0;
    }
    int free_here;
    block_scan(mine, sums, free_here);  // (and all threads are past the atomics)
    if (tid == 0) a.free_of[rank] = free_here;
    if (held) {
        for (int p = gtid; p < a.rows_in; p += gthreads) {
            a.children[p] = children[p];
            a.eldest[p] = eldest[p];
        }
    }
    // New pages that each row wants: all it needs, a thread to a row; a parent's first row
    // keeps what it can, a warp to a parent.
    for (int i = gtid; i < a.rows_out; i += gthreads) {
        const Row r = row_of(a, i, held ? eldest : a.eldest);
        const int n = max(r.need - r.full, 0);
        if (!r.eldest) a.wants[i] = n | (n > 0 && r.L % a.P != 0 ? 1 << 30 : 0);
    }
    for (int p = gwarp; p < a.rows_in; p += gwarps) {
        const int i = held ? eldest[p] : __ldcg(a.eldest + p);
        if (i >= a.rows_out) continue;  // (nobody continues it)
        const Row r = row_of(a, i, held ? eldest : a.eldest);
        int n = 0;
        bool copy = false;
        for (int s0 = r.full; s0 < r.need; s0 += 32) {
            const int s = s0 + lane;
            const bool fresh =
                s < r.need && !keeps(a, r, a.table[static_cast<size_t>(p) * a.max_pages + s]);
            copy |= fresh && s == r.full && r.L % a.P != 0;
            n += __popc(__ballot_sync(kFull, fresh));
        }
        copy = __any_sync(kFull, copy);
        if (lane == 0) a.wants[i] = n | (copy ? 1 << 30 : 0);
    }
    ptx::cluster_sync();

    // Where each row's new pages begin, and the free pages themselves.
    int total = 0, copies = 0;
    for (int i0 = 0; i0 < a.rows_out; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const int w = i < a.rows_out ? __ldcg(a.wants + i) : 0;
        int sum, sum_c;
        const int before = block_scan(w & 0x3fffffff, sums, sum);
        const int before_c = block_scan(w >> 30, sums, sum_c);
        if (rank == 0 && i < a.rows_out) {
            a.base[i] = total + before;
            a.copies[i] = copies + before_c;
        }
        total += sum;
        copies += sum_c;
    }
    int at = 0, free_all = 0;
    for (int r = 0; r < ctas; ++r) {
        const int f = __ldcg(a.free_of + r);
        at += r < rank ? f : 0;
        free_all += f;
    }
    constexpr int kEach = 4;
    for (int p0 = lo; p0 < hi && at < total; p0 += kEach * kPlanThreads) {
        bool is[kEach];
        int n = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int p = p0 + tid * kEach + j;
            is[j] = p < hi && a.refs[p] == 0;
            n += is[j];
        }
        int sum;
        int k = at + block_scan(n, sums, sum);
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (is[j] && k < total) a.list[k] = p0 + tid * kEach + j;
            k += is[j];
        }
        at += sum;
    }
    if (gtid == 0) {
        *a.count = copies;
        *a.free_all = free_all;
        if (total > free_all) report(a.status, TREE_ATTN_STATUS_NO_PAGE);
    }
    ptx::cluster_sync();

    // Lengths, and the pages that are copied.
    for (int i = gtid; i < a.rows_out; i += gthreads) {
        const Row r = row_of(a, i, held ? eldest : a.eldest);
        int L = r.L;
        if (__ldcg(a.wants + i) >> 30 != 0) {  // its first new page takes tokens
            const int k = __ldcg(a.base + i), c = __ldcg(a.copies + i);
            const int to = k < free_all ? __ldcg(a.list + k) : -1;
            const int from = a.table[static_cast<size_t>(r.parent) * a.max_pages + r.full];
            const bool ok = entry_ok(from, a.num_pages);
            if (!ok) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            a.copy_src[c] = ok && to >= 0 ? from : -1;
            a.copy_dst[c] = to;
            if (to < 0) L = r.full * a.P;  // the tokens that found no page
        }
        a.lens_out[i] = L;
    }
}

// The plan as the first kernel left it in the workspace.
struct Stored {
    const ForkArgs& a;
    const int32_t* eldest;
    __device__ __forceinline__ explicit Stored(const ForkArgs& args) : a(args), eldest(args.eldest) {}
    __device__ __forceinline__ int base(int i) const { return a.base[i]; }
    __device__ __forceinline__ int free_all() const { return *a.free_all; }
    __device__ __forceinline__ int free_at(int k) const { return a.list[k]; }
    __device__ __forceinline__ int children(int p) const { return a.children[p]; }
};

// One warp: row i of the new table (TABLE), and the counts of its own pages in refs (REFS).
template <bool TABLE, bool REFS, typename Plan>
__device__ __forceinline__ void fork_row(const ForkArgs& a, const Plan& plan, int i, int32_t* refs) {
    const int lane = threadIdx.x & 31;
    const Row r = row_of(a, i, plan.eldest);
    const int32_t* from = a.table + static_cast<size_t>(max(r.parent, 0)) * a.max_pages;
    int32_t* to = a.table_out + static_cast<size_t>(i) * a.max_pages;
    int next = plan.base(i);
    const int free_all = plan.free_all();
    if (TABLE) {
#pragma unroll 4
        for (int s = lane; s < a.max_pages; s += 32) {  // the shared ones
            if (s >= r.full && s < r.need) continue;
            int e = s < r.full ? from[s] : -1;
            if (s < r.full && !entry_ok(e, a.num_pages)) {
                report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                e = -1;
            }
            to[s] = e;
        }
        __syncwarp();
    }
    for (int s0 = r.full; s0 < r.need; s0 += 32) {
        const int s = s0 + lane;
        int e = s < r.need && r.parent >= 0 ? from[s] : -1;
        const bool fresh = s < r.need && !keeps(a, r, e);
        const unsigned who = __ballot_sync(kFull, fresh);
        if (fresh) {
            const int k = next + __popc(who & ((1u << lane) - 1u));
            e = k < free_all ? plan.free_at(k) : -1;
        }
        if (s < r.need) {
            if (REFS && e >= 0) atomicAdd(refs + e, 1);
            if (TABLE) to[s] = e;
        }
        next += __popc(who);
    }
}

// One warp: the counts, in refs, of what row p had.
template <typename Plan>
__device__ __forceinline__ void fork_release(const ForkArgs& a, const Plan& plan, int p,
                                             int32_t* refs) {
    bool bad;
    const int L = clamp_seq_len(a.lens[p], a.P, a.max_pages, bad);
    const int full = bad ? 0 : L / a.P;
    const int kept = plan.children(p) - 1;  // for shared pages
    const int32_t* from = a.table + static_cast<size_t>(p) * a.max_pages;
#pragma unroll 4
    for (int s = (kept == 0 ? full : 0) + (threadIdx.x & 31); s < a.max_pages; s += 32) {
        const int e = from[s];
        if (entry_ok(e, a.num_pages))
            atomicAdd(refs + e, s < full ? kept : -1);
        else if (e != -1)
            report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
    }
}

// ---------------------------------------------------------------------------
// Compact.  With u(p) = used pages before p and n the used pages in all, the
// k-th used page at or past n goes to the k-th free page before n:
//   page p >= n is mover u(p) - u(n), page p < n is hole p - u(p).
// ---------------------------------------------------------------------------
struct CompactArgs {
    const int32_t* table;
    const int32_t* refs;
    int32_t* table_out;
    int32_t* refs_out;
    int32_t* n_used;  // [1]
    long long entries;
    int num_pages;
    // workspace
    int32_t* copy_src;  // [num_pages]
    int32_t* copy_dst;  // [num_pages]
    int32_t* count;     // [1]
    int32_t* used_of;   // [kMaxCtas]
    int32_t* before_n;  // [1] u(n)
    int32_t* movers;    // [num_pages], at u(p)
    int32_t* to;        // [num_pages] new place of a page that moves
    int32_t* status;
};

__global__ void __launch_bounds__(kPlanThreads) compact_kernel(const CompactArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ int sums[kPlanWarps];
    const int tid = threadIdx.x;
    const int ctas = static_cast<int>(ptx::cluster_size());
    const int rank = static_cast<int>(ptx::cluster_rank());
    const int gtid = rank * kPlanThreads + tid, gthreads = ctas * kPlanThreads;
    int lo, hi;
    my_pages(a.num_pages, lo, hi);

    int mine = 0;
    for (int p = lo + tid; p < hi; p += kPlanThreads) mine += a.refs[p] > 0;
    int used_here;
    block_scan(mine, sums, used_here);
    if (tid == 0) a.used_of[rank] = used_here;
    ptx::cluster_sync();

    int u0 = 0, n = 0;
    for (int r = 0; r < ctas; ++r) {
        const int c = __ldcg(a.used_of + r);
        u0 += r < rank ? c : 0;
        n += c;
    }
    if (gtid == 0 && n == a.num_pages) *a.before_n = n;
    constexpr int kEach = 4;
    for (int p0 = lo; p0 < hi; p0 += kEach * kPlanThreads) {
        int c[kEach], m = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int p = p0 + tid * kEach + j;
            c[j] = p < hi ? a.refs[p] : 0;
            m += c[j] > 0;
        }
        int sum;
        int u = u0 + block_scan(m, sums, sum);
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int p = p0 + tid * kEach + j;
            if (p >= hi) break;
            if (p == n) *a.before_n = u;
            if (p < n) {
                if (c[j] > 0)
                    a.refs_out[p] = c[j];
                else
                    a.copy_dst[p - u] = p;
            } else {
                a.refs_out[p] = 0;
                if (c[j] > 0) a.movers[u] = p;
            }
            u += c[j] > 0;
        }
        u0 += sum;
    }
    ptx::cluster_sync();

    const int un = __ldcg(a.before_n);
    const int moves = n - un;
    for (int k = gtid; k < moves; k += gthreads) {
        const int from = __ldcg(a.movers + un + k), to = __ldcg(a.copy_dst + k);
        a.copy_src[k] = from;
        a.to[from] = to;
        a.refs_out[to] = a.refs[from];
    }
    if (gtid == 0) {
        *a.count = moves;
        *a.n_used = n;
    }
}

// The pages' new places in the table, by all warps of the copies' grid.
__device__ __forceinline__ void compact_table(const CompactArgs& a, long long thread,
                                              long long threads) {
    if (thread >= a.entries) return;
    const int n = *a.n_used;
    for (long long i = thread; i < a.entries; i += threads) {
        int e = a.table[i];
        if (e != -1) {
            if (!entry_ok(e, a.num_pages) || a.refs[e] <= 0) {
                report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                e = -1;
            } else if (e >= n) {
                e = a.to[e];
            }
        }
        a.table_out[i] = e;
    }
}

// ---------------------------------------------------------------------------
// Copies: page src[k] of every pool to its page dst[k].  A warp moves 4 KB at a
// time, eight 16-byte vectors to a lane, all loaded before the first is stored.
// ---------------------------------------------------------------------------
constexpr int kPoolsMost = 120;  // of one launch
constexpr int kPiece = 4096;     // bytes a warp moves at a time
constexpr int kCopyThreads = 256;

struct CopyArgs {
    uint8_t* pool[kPoolsMost];
    long long bytes[kPoolsMost];  // of one page
    int first[kPoolsMost + 1];    // first piece of each pool within a page's
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;  // nullable: n
    int n, n_pools, num_pages;
    int32_t* status;
};

__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// What is done beside the copies: nothing, or the table of a fork or a compaction.
struct NoTable {};

// All pairs k < n of a launch, spread over the grid's warps: pair_of(k, src, dst) says which.
template <typename PairOf>
__device__ __forceinline__ void copy_pairs(const CopyArgs& a, int n, PairOf pair_of) {
    if (a.n_pools == 0) return;
    const int lane = threadIdx.x & 31;
    const int per = a.first[a.n_pools];
    const int warps = gridDim.x * (kCopyThreads / 32);
    const int step_k = warps / per, step_c = warps % per;
    const int w0 = blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32;
    int k = w0 / per, c = w0 % per;
    while (k < n) {
        int s, d;
        pair_of(k, s, d);
        if (s >= 0 && d >= 0 && s < a.num_pages && d < a.num_pages) {
            int lo = 0, hi = a.n_pools - 1;  // the pool that piece c belongs to
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.first[mid] <= c)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const long long page = a.bytes[lo];
            const long long at = static_cast<long long>(c - a.first[lo]) * kPiece;
            const int m = static_cast<int>(min(page - at, static_cast<long long>(kPiece)));
            const uint8_t* from = a.pool[lo] + s * page + at;
            uint8_t* to = a.pool[lo] + d * page + at;
            if (((page | reinterpret_cast<uintptr_t>(a.pool[lo])) & 15) == 0) {
                uint4 v[kPiece / 512];
#pragma unroll
                for (int i = 0; i < kPiece / 512; ++i)
                    if (i * 512 + lane * 16 < m) v[i] = ld_once(from + i * 512 + lane * 16);
#pragma unroll
                for (int i = 0; i < kPiece / 512; ++i)
                    if (i * 512 + lane * 16 < m)
                        *reinterpret_cast<uint4*>(to + i * 512 + lane * 16) = v[i];
            } else {
                for (int i = lane; i < m; i += 32) to[i] = from[i];
            }
        } else if (lane == 0 && (s < -1 || d < -1 || s >= a.num_pages || d >= a.num_pages)) {
            report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
        }
        k += step_k;
        c += step_c;
        if (c >= per) {
            c -= per;
            ++k;
        }
    }
}

template <typename Table>
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ CopyArgs a, const __grid_constant__ Table f) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if constexpr (std::is_same<Table, CompactArgs>::value) {
        compact_table(f, static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x,
                      static_cast<long long>(gridDim.x) * kCopyThreads);
    }
    if constexpr (std::is_same<Table, ForkArgs>::value) {
        const int warps = gridDim.x * (kCopyThreads / 32);
        // (from the last warp on: the first ones have the most copies)
        for (int i = warps - 1 - (blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32);
             i < f.rows_out + f.rows_in; i += warps) {
            if (i < f.rows_out)
                fork_row<true, true>(f, Stored(f), i, f.refs_out);
            else
                fork_release(f, Stored(f), i - f.rows_out, f.refs_out);
        }
    }
    copy_pairs(a, a.count != nullptr ? min(max(*a.count, 0), a.n) : a.n, [&](int k, int& s, int& d) {
        s = a.src[k];
        d = a.dst[k];
    });
}

// ---------------------------------------------------------------------------
// Few pages: which of them are used (free) fits into one bit each, and any CTA finds from
// those bits and the counts before each 32 of them, by bisection, the k-th of them.  So
// every CTA of the copies makes the whole plan for itself, and nothing waits for another.
// Compaction: 256 pages of 128 KB, 100 used, 10.3 us for 14.4 with a plan of its own; 2048
// pages, 262 MB moved, 52 for 56; 4096 pages, whose counts take every CTA longer to read,
// 95 for 91.
// ---------------------------------------------------------------------------
constexpr int kFewWords = 64;
constexpr int kFewPages = 32 * kFewWords;
constexpr int kCopyWarps = kCopyThreads / 32;
static_assert(kFewWords <= kCopyThreads, "a thread counts a word");

// Place of the r-th set bit of w.
__device__ __forceinline__ int nth_bit(uint32_t w, int r) {
    int at = 0;
#pragma unroll
    for (int half = 16; half > 0; half >>= 1) {
        const int c = __popc(w & ((1u << half) - 1u));
        if (r >= c) {
            r -= c;
            w >>= half;
            at += half;
        }
    }
    return at;
}

struct Bitmap {  // in shared memory
    uint32_t bits[kFewWords];
    int before[kFewWords];  // marked pages before those of a word
    int sums[kCopyWarps];
    int words;

    // By all threads: marks the pages that `is` says; how many there are.
    template <typename Is>
    __device__ __forceinline__ int make(int num_pages, Is is) {
        const int tid = threadIdx.x, lane = tid & 31;
        const int n_words = (num_pages + 31) / 32;
#pragma unroll 8
        for (int w = tid >> 5; w < n_words; w += kCopyWarps) {
            const int p = 32 * w + lane;
            const unsigned m = __ballot_sync(kFull, p < num_pages && is(p));
            if (lane == 0) bits[w] = m;
        }
        __syncthreads();
        int n;
        const int earlier = block_scan<kCopyWarps>(tid < n_words ? __popc(bits[tid]) : 0, sums, n);
        if (tid < kFewWords) before[tid] = earlier;
        if (tid == 0) words = n_words;
        __syncthreads();
        return n;
    }
    __device__ __forceinline__ bool has(int p) const { return (bits[p / 32] >> p % 32 & 1u) != 0; }
    __device__ __forceinline__ int marked_before(int p) const {
        return before[p / 32] + __popc(bits[p / 32] & ((1u << p % 32) - 1u));
    }
    __device__ __forceinline__ int marked_at(int r) const {  // the r-th marked page
        int w = 0;
#pragma unroll
        for (int step = kFewWords / 2; step > 0; step >>= 1)
            if (w + step < words && before[w + step] <= r) w += step;
        return 32 * w + nth_bit(bits[w], r - before[w]);
    }
    __device__ __forceinline__ int unmarked_at(int r) const {  // the r-th other page
        int w = 0;
#pragma unroll
        for (int step = kFewWords / 2; step > 0; step >>= 1)
            if (w + step < words && 32 * (w + step) - before[w + step] <= r) w += step;
        return 32 * w + nth_bit(~bits[w], r - (32 * w - before[w]));
    }
};

__global__ void __launch_bounds__(kCopyThreads, 4)
    compact_few_kernel(const __grid_constant__ CopyArgs a, const __grid_constant__ CompactArgs f) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ Bitmap used;
    const int tid = threadIdx.x;
    const int n = used.make(f.num_pages, [&](int p) { return f.refs[p] > 0; });
    const int un = n == f.num_pages ? n : used.marked_before(n);
    if (f.refs_out != nullptr) {  // (the first of several launches)
        const long long thread = static_cast<long long>(blockIdx.x) * kCopyThreads + tid;
        const long long threads = static_cast<long long>(gridDim.x) * kCopyThreads;
        if (thread == 0) *f.n_used = n;
        for (long long i = thread; i < f.num_pages; i += threads) {
            const int p = static_cast<int>(i);
            int from = p;
            if (p < n && !used.has(p)) from = used.marked_at(un + p - used.marked_before(p));
            f.refs_out[p] = p < n ? f.refs[from] : 0;
        }
        for (long long i = thread; i < f.entries; i += threads) {
            int e = f.table[i];
            if (e != -1) {
                if (!entry_ok(e, f.num_pages) || !used.has(e)) {
                    report(f.status, TREE_ATTN_STATUS_BAD_PAGE);
                    e = -1;
                } else if (e >= n) {
                    e = used.unmarked_at(used.marked_before(e) - un);
                }
            }
            f.table_out[i] = e;
        }
    }
    copy_pairs(a, n - un, [&](int k, int& s, int& d) {
        s = used.marked_at(un + k);
        d = used.unmarked_at(k);
    });
}

// Fork, of few rows and pages: the last CTA also keeps the counts, in shared memory.  Against
// a plan of its own, three runs of each, 2048 pages in all: 16 rows with tables of 128
// entries 7.0 to 8.3 us and 8.4 to 10.4, of 2048 entries 14.5 and 18.6; 32 rows of 64 entries
// 12.3 and 10.4, of 128 entries 10.4 to 10.8 and 10.4, of 2048 entries 24.7 and 20.6.
constexpr int kFewRows = 16;

struct FewRows {
    int children_of[kFewRows], eldest[kFewRows], base_of[kFewRows];
    int wants[kFewRows], tokens[kFewRows];
    int src_of[kFewRows];  // the page that holds the last tokens of a row's parent
    int src[kFewRows], dst[kFewRows];
    int n_free, n_copies;
    int refs[kFewPages];
    Bitmap free;
    __device__ __forceinline__ int base(int i) const { return base_of[i]; }
    __device__ __forceinline__ int free_all() const { return n_free; }
    __device__ __forceinline__ int free_at(int k) const { return free.marked_at(k); }
    __device__ __forceinline__ int children(int p) const { return children_of[p]; }
};

__global__ void __launch_bounds__(kCopyThreads, 4)
    fork_few_kernel(const __grid_constant__ CopyArgs c, const __grid_constant__ ForkArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __shared__ FewRows sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool first = a.table_out != nullptr || a.rows_out == 0;  // (of several launches)
    if (tid < kFewRows) {
        sm.children_of[tid] = 0;
        sm.eldest[tid] = 0x7fffffff;
    }
    __syncthreads();
    if (tid < a.rows_out) {
        const int p = a.src[tid];
        if (p >= 0 && p < a.rows_in) {
            atomicAdd(sm.children_of + p, 1);
            atomicMin(sm.eldest + p, tid);
        }
    }
    const int n_free = sm.free.make(a.num_pages, [&](int p) { return a.refs[p] == 0; });
    if (tid == 0) sm.n_free = n_free;
    // New pages of each row, and whether one is a copy.
    for (int i = warp; i < a.rows_out; i += kCopyWarps) {
        const Row r = row_of(a, i, sm.eldest);
        const int32_t* from = a.table + static_cast<size_t>(max(r.parent, 0)) * a.max_pages;
        int n = 0, e_full = -1;
        bool copy = false;
        for (int s0 = r.full; s0 < r.need; s0 += 32) {
            const int s = s0 + lane;
            const int e = s < r.need && r.parent >= 0 ? from[s] : -1;
            const bool fresh = s < r.need && !keeps(a, r, e);
            n += __popc(__ballot_sync(kFull, fresh));
            if (s == r.full) {  // (lane 0)
                copy = fresh && r.L % a.P != 0;
                e_full = e;
            }
        }
        if (lane == 0) {
            sm.wants[i] = n | (copy ? 1 << 30 : 0);
            sm.tokens[i] = r.L;
            sm.src_of[i] = e_full;
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int wants = lane < a.rows_out ? sm.wants[lane] : 0;
        const int n = wants & 0x3fffffff;
        const bool copy = wants >> 30 != 0;
        int upto = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(kFull, upto, off);
            if (lane >= off) upto += y;
        }
        const int total = __shfl_sync(kFull, upto, 31);
        const unsigned who = __ballot_sync(kFull, copy);
        if (lane < a.rows_out) {
            const int k = upto - n;
            int L = sm.tokens[lane];
            sm.base_of[lane] = k;
            if (copy) {  // its first new page takes tokens
                const int at = __popc(who & ((1u << lane) - 1u)), e = sm.src_of[lane];
                const int to = k < n_free ? sm.free.marked_at(k) : -1;
                const bool ok = entry_ok(e, a.num_pages);
                if (!ok) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
                sm.src[at] = ok && to >= 0 ? e : -1;
                sm.dst[at] = to;
                if (to < 0) L -= L % a.P;  // the tokens that found no page
            }
            if (first && blockIdx.x == 0) a.lens_out[lane] = L;
        }
        if (lane == 0) {
            sm.n_copies = __popc(who);
            if (total > n_free) report(a.status, TREE_ATTN_STATUS_NO_PAGE);
        }
    }
    __syncthreads();
    if (first) {
        const int warps = gridDim.x * kCopyWarps;
        for (int i = blockIdx.x * kCopyWarps + warp; i < a.rows_out; i += warps)
            fork_row<true, false>(a, sm, i, nullptr);
        if (blockIdx.x == gridDim.x - 1) {
            for (int p = tid; p < a.num_pages; p += kCopyThreads) sm.refs[p] = a.refs[p];
            __syncthreads();
            for (int i = warp; i < a.rows_out; i += kCopyWarps)
                fork_row<false, true>(a, sm, i, sm.refs);
            for (int p = warp; p < a.rows_in; p += kCopyWarps) fork_release(a, sm, p, sm.refs);
            __syncthreads();
            for (int p = tid; p < a.num_pages; p += kCopyThreads) a.refs_out[p] = sm.refs[p];
        }
    }
    copy_pairs(c, sm.n_copies, [&](int k, int& s, int& d) {
        s = sm.src[k];
        d = sm.dst[k];
    });
}

// ---------------------------------------------------------------------------

int rc_of(cudaError_t e) { return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA; }

int check_pools(void* const* pools, const size_t* page_bytes, int n_pools) {
    if (n_pools < 0) return TREE_ATTN_ERR_SHAPE;
    if (n_pools == 0) return TREE_ATTN_OK;
    if (!pools || !page_bytes) return TREE_ATTN_ERR_NULL;
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i]) return TREE_ATTN_ERR_NULL;
        if (page_bytes[i] < 1 || page_bytes[i] > (static_cast<size_t>(1) << 31))
            return TREE_ATTN_ERR_SHAPE;
    }
    return TREE_ATTN_OK;
}

// Pools in launches of at most kPoolsMost, launch(grid, pools, whether it is the first),
// of n pages each; the first also makes a table (whose rows, or entries, take `more` warps).
// As many CTAs as the SMs hold at once (`each`) take the pieces in turn.
template <typename Launch>
int enqueue_copies(void* const* pools, const size_t* page_bytes, int n_pools, const int32_t* src,
                   const int32_t* dst, const int32_t* count, int n, int num_pages, int32_t* status,
                   int each, long long more, Launch launch) {
    if (n == 0 && more == 0) return TREE_ATTN_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TREE_ATTN_ERR_CUDA;
    const int sms = sms_of(dev);
    if (sms == 0) return TREE_ATTN_ERR_CUDA;
    CopyArgs a;
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.n = n;
    a.num_pages = num_pages;
    a.status = status;
    for (int i = 0; i < n_pools || more > 0;) {
        long long pieces = 0;
        int m = 0;
        for (; i < n_pools && m < kPoolsMost; ++i, ++m) {
            const long long of_page = (static_cast<long long>(page_bytes[i]) + kPiece - 1) / kPiece;
            if (m > 0 && pieces + of_page > (1LL << 30)) break;
            a.pool[m] = static_cast<uint8_t*>(pools[i]);
            a.bytes[m] = static_cast<long long>(page_bytes[i]);
            a.first[m] = static_cast<int>(pieces);
            pieces += of_page;
        }
        a.first[m] = static_cast<int>(pieces);
        a.n_pools = m;
        long long warps = pieces * n;
        if (warps < more) warps = more;
        const long long ctas = (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
        const long long most = static_cast<long long>(each) * sms;
        const int grid = static_cast<int>(ctas < most ? ctas : most);
        if (grid == 0) return TREE_ATTN_OK;
        const int rc = rc_of(launch(dim3(grid), a, more > 0));
        if (rc != TREE_ATTN_OK) return rc;
        more = 0;  // (it is made once)
    }
    return TREE_ATTN_OK;
}

// One CTA where the whole plan is little work, else a cluster.
int plan_ctas(long long work) { return work <= 8192 ? 1 : kMaxCtas; }

bool pages_shape_ok(int rows, int max_pages, int num_pages) {
    return rows >= 0 && rows < (1 << 24) && max_pages >= 1 && num_pages >= 1 &&
           max_pages < (1 << 30) && num_pages < (1 << 30) &&
           static_cast<long long>(rows) * max_pages < (1LL << 31);  // (new pages are counted in ints)
}

size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }

bool few_rows(int rows_in, int rows_out, int num_pages) {
    return rows_in <= kFewRows && rows_out <= kFewRows && num_pages <= kFewPages;
}

size_t fork_bytes(int rows_in, int rows_out, int num_pages) {
    if (few_rows(rows_in, rows_out, num_pages)) return 0;
    return padded((64 + 2 * static_cast<size_t>(rows_in) + 5 * static_cast<size_t>(rows_out) +
                   static_cast<size_t>(num_pages)) * 4);
}
size_t compact_bytes(int num_pages) {
    return num_pages <= kFewPages ? 0 : padded((64 + 4 * static_cast<size_t>(num_pages)) * 4);
}

}  // namespace
}  // namespace treeattn

using namespace treeattn;

extern "C" {

int tree_kv_copy_pages(void* const* pools, const size_t* page_bytes, int n_pools,
                       const int32_t* src, const int32_t* dst, const int32_t* count, int n,
                       int num_pages, int32_t* status, void* stream) {
    if (n < 0 || n >= (1 << 30) || num_pages < 1 || num_pages >= (1 << 30))
        return TREE_ATTN_ERR_SHAPE;
    const int rc = check_pools(pools, page_bytes, n_pools);
    if (rc != TREE_ATTN_OK) return rc;
    if (n == 0 || n_pools == 0) return TREE_ATTN_OK;
    if (!src || !dst) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(src, 4) || !ptr_aligned(dst, 4) || !ptr_aligned(count, 4) ||
        !ptr_aligned(status, 4))
        return TREE_ATTN_ERR_ALIGN;
    return enqueue_copies(pools, page_bytes, n_pools, src, dst, count, n, num_pages, status, 8, 0,
                          [&](dim3 grid, const CopyArgs& a, bool) {
                              return launch_dependent(copy_kernel<NoTable>, grid,
                                                      dim3(kCopyThreads), 0,
                                                      static_cast<cudaStream_t>(stream), a,
                                                      NoTable());
                          });
}

size_t tree_kv_fork_workspace_size(int rows_in, int rows_out, int num_pages) {
    if (rows_in < 0 || rows_out < 0 || num_pages < 1) return 0;
    return fork_bytes(rows_in, rows_out, num_pages);
}

int tree_kv_fork(void* const* pools, const size_t* page_bytes, int n_pools,
                 const int32_t* block_table, int max_pages_per_seq, const int32_t* seq_lens,
                 const int32_t* page_refs, const int32_t* src, const int32_t* reserve,
                 int reserve_all, int32_t* block_table_out, int32_t* seq_lens_out,
                 int32_t* page_refs_out, int rows_in, int rows_out, int page_size, int num_pages,
                 void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    if (!pages_shape_ok(rows_in, max_pages_per_seq, num_pages) ||
        !pages_shape_ok(rows_out, max_pages_per_seq, num_pages) || !page_size_ok(page_size) ||
        reserve_all < 0)
        return TREE_ATTN_ERR_SHAPE;
    const int rc = check_pools(pools, page_bytes, n_pools);
    if (rc != TREE_ATTN_OK) return rc;
    if (!page_refs || !page_refs_out || (rows_in > 0 && (!block_table || !seq_lens)) ||
        (rows_out > 0 && (!src || !block_table_out || !seq_lens_out)))
        return TREE_ATTN_ERR_NULL;
    if (page_refs_out == page_refs || (rows_out > 0 && block_table_out == block_table) ||
        (rows_out > 0 && seq_lens_out == seq_lens))
        return TREE_ATTN_ERR_SHAPE;
    const void* ints[] = {block_table, seq_lens,     page_refs,     src,   reserve,
                          status,      seq_lens_out, page_refs_out, block_table_out};
    for (const void* p : ints)
        if (!ptr_aligned(p, 4)) return TREE_ATTN_ERR_ALIGN;
    const size_t bytes = fork_bytes(rows_in, rows_out, num_pages);
    if (bytes > 0 && (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < bytes))
        return TREE_ATTN_ERR_WORKSPACE;
    ForkArgs a = {};
    a.table = block_table;
    a.lens = seq_lens;
    a.refs = page_refs;
    a.src = src;
    a.reserve = reserve;
    a.reserve_all = reserve_all;
    a.table_out = block_table_out;
    a.lens_out = seq_lens_out;
    a.refs_out = page_refs_out;
    a.rows_in = rows_in;
    a.rows_out = rows_out;
    a.max_pages = max_pages_per_seq;
    a.P = page_size;
    a.num_pages = num_pages;
    a.status = status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long more = static_cast<long long>(rows_in) + rows_out;
    if (few_rows(rows_in, rows_out, num_pages))
        return enqueue_copies(pools, page_bytes, n_pools, nullptr, nullptr, nullptr, rows_out,
                              num_pages, status, 4, more > 0 ? more : 1,
                              [&](dim3 grid, const CopyArgs& c, bool first) {
                                  if (!first) a.table_out = nullptr;
                                  return launch_dependent(fork_few_kernel, grid,
                                                          dim3(kCopyThreads), 0, s, c, a);
                              });
    int32_t* w = static_cast<int32_t*>(workspace);
    a.count = w;
    a.free_all = w + 1;
    a.free_of = w + 32;
    w += 64;
    a.children = w;
    a.eldest = w + rows_in;
    w += 2 * static_cast<size_t>(rows_in);
    a.copy_src = w;
    a.copy_dst = w + rows_out;
    w += 2 * static_cast<size_t>(rows_out);
    a.wants = w;
    a.base = w + rows_out;
    w += 2 * static_cast<size_t>(rows_out);
    a.copies = w;
    a.list = w + rows_out;
    const long long work =
        num_pages + static_cast<long long>(rows_in + rows_out) * max_pages_per_seq;
    const int ctas = plan_ctas(work);
    const int rp = rc_of(launch_cluster(fork_kernel, dim3(ctas), dim3(kPlanThreads), 0, ctas, s, a));
    if (rp != TREE_ATTN_OK) return rp;
    return enqueue_copies(
        pools, page_bytes, n_pools, a.copy_src, a.copy_dst, a.count, rows_out, num_pages, status, 8,
        more, [&](dim3 grid, const CopyArgs& c, bool first) {
            return first ? launch_dependent(copy_kernel<ForkArgs>, grid, dim3(kCopyThreads), 0, s,
                                            c, a)
                         : launch_dependent(copy_kernel<NoTable>, grid, dim3(kCopyThreads), 0, s, c,
                                            NoTable());
        });
}

size_t tree_kv_compact_workspace_size(int num_pages) {
    return num_pages < 1 ? 0 : compact_bytes(num_pages);
}

int tree_kv_compact(void* const* pools, const size_t* page_bytes, int n_pools,
                    const int32_t* block_table, int max_pages_per_seq, const int32_t* page_refs,
                    int32_t* block_table_out, int32_t* page_refs_out, int32_t* n_used, int rows,
                    int num_pages, void* workspace, size_t workspace_bytes, int32_t* status,
                    void* stream) {
    if (!pages_shape_ok(rows, max_pages_per_seq, num_pages)) return TREE_ATTN_ERR_SHAPE;
    const int rc = check_pools(pools, page_bytes, n_pools);
    if (rc != TREE_ATTN_OK) return rc;
    if (!page_refs || !page_refs_out || !n_used ||
        (rows > 0 && (!block_table || !block_table_out)))
        return TREE_ATTN_ERR_NULL;
    if (page_refs_out == page_refs) return TREE_ATTN_ERR_SHAPE;
    const void* ints[] = {block_table, page_refs, block_table_out, page_refs_out, n_used, status};
    for (const void* p : ints)
        if (!ptr_aligned(p, 4)) return TREE_ATTN_ERR_ALIGN;
    const size_t need = compact_bytes(num_pages);
    if (need > 0 && (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < need))
        return TREE_ATTN_ERR_WORKSPACE;
    CompactArgs a = {};
    a.table = block_table;
    a.refs = page_refs;
    a.table_out = block_table_out;
    a.refs_out = page_refs_out;
    a.n_used = n_used;
    a.entries = static_cast<long long>(rows) * max_pages_per_seq;
    a.num_pages = num_pages;
    a.status = status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long more = (a.entries + 127) / 128;
    if (num_pages <= kFewPages)
        return enqueue_copies(pools, page_bytes, n_pools, nullptr, nullptr, nullptr, num_pages / 2,
                              num_pages, status, 4, more > 0 ? more : 1,
                              [&](dim3 grid, const CopyArgs& c, bool first) {
                                  if (!first) a.refs_out = nullptr;
                                  return launch_dependent(compact_few_kernel, grid,
                                                          dim3(kCopyThreads), 0, s, c, a);
                              });
    int32_t* w = static_cast<int32_t*>(workspace);
    a.count = w;
    a.before_n = w + 1;
    a.used_of = w + 32;
    w += 64;
    a.copy_src = w;
    a.copy_dst = w + num_pages;
    w += 2 * static_cast<size_t>(num_pages);
    a.movers = w;
    a.to = w + num_pages;
    const int ctas = plan_ctas(num_pages + a.entries);
    const int rp =
        rc_of(launch_cluster(compact_kernel, dim3(ctas), dim3(kPlanThreads), 0, ctas, s, a));
    if (rp != TREE_ATTN_OK) return rp;
    return enqueue_copies(
        pools, page_bytes, n_pools, a.copy_src, a.copy_dst, a.count, num_pages / 2, num_pages,
        status, 8, more, [&](dim3 grid, const CopyArgs& c, bool first) {
            return first ? launch_dependent(copy_kernel<CompactArgs>, grid, dim3(kCopyThreads), 0,
                                            s, c, a)
                         : launch_dependent(copy_kernel<NoTable>, grid, dim3(kCopyThreads), 0, s, c,
                                            NoTable());
        });
}

}  // extern "C"
