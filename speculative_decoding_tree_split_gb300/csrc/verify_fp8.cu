// verify_fp8.cu -- split tree attention over the 8-bit paged cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/tree_attn.h"
#include "fp8.cuh"
#include "kernels.cuh"
#include "launch.cuh"
#include "layout.h"
#include "ptx.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

struct Fp8Args {
    const uint16_t* q;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const uint8_t* k_scales;
    const uint8_t* v_scales;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const uint16_t* tree_k;
    const uint16_t* tree_v;
    const uint64_t* mask;
    int mask_stride;
    const int32_t* parents;
    int parents_stride;
    uint64_t* mask_out;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int B, Hq, Hkv, G, T, P, max_pages, num_pages;
    float scale_log2;
};

// One warp per (sequence, tree node, query head): a running softmax over the
// committed rows and then the tree rows.
template <int D>
__global__ void __launch_bounds__(128) verify_fp8_rows_kernel(const Fp8Args a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(a.B) * a.T * a.Hq) return;
    const int h = static_cast<int>(w % a.Hq);
    const int t = static_cast<int>(w / a.Hq % a.T);
    const int b = static_cast<int>(w / a.Hq / a.T);
    const int hk = h / a.G;
    bool bad;
    const int L = clamp_seq_len(a.seq_lens[b], a.P, a.max_pages, bad);
    if (bad && lane == 0) report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    uint64_t bits = 0;
    if (a.parents != nullptr) {
        const int32_t* par = a.parents + static_cast<size_t>(b) * a.parents_stride;
        for (int node = t; node >= 0;) {
            bits |= 1ull << node;
            const int up = par[node];
            if (up < -1 || up >= node) {
                report(a.status, TREE_ATTN_STATUS_BAD_PARENT);
                break;
            }
            node = up;
        }
        if (h == 0 && lane == 0 && a.mask_out != nullptr && (a.parents_stride != 0 || b == 0))
            a.mask_out[static_cast<size_t>(b) * a.parents_stride + t] = bits;
    } else {
        bits = a.mask[static_cast<size_t>(b) * a.mask_stride + t];
        if (a.T < 64) bits &= (1ull << a.T) - 1ull;
    }
    auto bf = [](const uint16_t* p, int e) { return __uint_as_float(uint32_t(p[e]) << 16); };
    float q[E], acc[E], kv[E], vv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf(a.q + w * D, lane * E + e);
        acc[e] = 0.f;
    }
    float m = -__builtin_huge_valf(), l = 0.f;
    auto add_key = [&]() {
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(q[e], kv[e], x);
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
        x *= a.scale_log2;
        const float mn = fmaxf(m, x);
        if (mn == -__builtin_huge_valf()) return;
        const float al = exp2f(m - mn), p = exp2f(x - mn);
        l = l * al + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * al + p * vv[e];
        m = mn;
    };
    auto code = [](uint32_t c) {
        const uint32_t h2 = f16x2_of_e4m3x2(c);
        float f;
        asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo;}" : "=f"(f) : "r"(h2));
        return f;
    };
    for (int p = 0; p < L; ++p) {
        const int page = a.block_table[static_cast<size_t>(b) * a.max_pages + p / a.P];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) report(a.status, TREE_ATTN_STATUS_BAD_PAGE);
            continue;
        }
        const long long row = (static_cast<long long>(page) * a.Hkv + hk) * a.P + p % a.P;
        const float fk = scale_of(a.k_scales[row]), fv = scale_of(a.v_scales[row]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            kv[e] = code(a.k_pages[row * D + lane * E + e]) * fk;
            vv[e] = code(a.v_pages[row * D + lane * E + e]) * fv;
        }
        add_key();
    }
    for (int j = 0; j < a.T; ++j) {
        if (((bits >> j) & 1ull) == 0) continue;
        const long long row = (static_cast<long long>(b) * a.T + j) * a.Hkv + hk;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            kv[e] = bf(a.tree_k + row * D, lane * E + e);
            vv[e] = bf(a.tree_v + row * D, lane * E + e);
        }
        add_key();
    }
    const bool none = m == -__builtin_huge_valf();
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const __nv_bfloat16 o = __float2bfloat16_rn(none ? 0.f : acc[e] / l);
        a.out[w * D + lane * E + e] = *reinterpret_cast<const uint16_t*>(&o);
    }
    if (lane == 0) a.lse[w] = none ? m : (m + log2f(l)) * 0.69314718055994530942f;
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
    Fp8Args a;
    a.q = q;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.tree_k = tree_k;
    a.tree_v = tree_v;
    a.mask = mask;
    a.mask_stride = mask_stride;
    a.parents = parents;
    a.parents_stride = parents_stride;
    a.mask_out = mask_out;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.T = T;
    a.P = page_size;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
    const long long rows = static_cast<long long>(B) * T * Hq;
    const cudaError_t e = launch_dependent(
        d == 128 ? verify_fp8_rows_kernel<128> : verify_fp8_rows_kernel<64>,
        dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
        static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
