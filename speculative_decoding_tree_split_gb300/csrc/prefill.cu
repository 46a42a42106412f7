// prefill.cu -- causal attention over whole prompts of different lengths,
// packed one after the other, with grouped heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/tree_attn.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace treeattn {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

struct PrefillArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // token and head strides (elements)
    const int32_t* cu;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int B, N, Hq, Hkv, G;
    float scale_log2;
};

// One warp per (token, query head): a running softmax over the tokens of the
// sequence up to its own.
template <int D>
__global__ void __launch_bounds__(128) prefill_rows_kernel(const PrefillArgs a) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += 128)
            if (a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.N)
                report(a.status, TREE_ATTN_STATUS_BAD_SEQ_LEN);
    if (w >= static_cast<long long>(a.N) * a.Hq) return;
    const int i = static_cast<int>(w / a.Hq), h = static_cast<int>(w % a.Hq), hk = h / a.G;
    int lo = 0, hi = a.B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo >= a.B || a.cu[lo] < 0 || a.cu[lo] > i || i >= a.cu[lo + 1] || a.cu[lo + 1] > a.N) return;
    auto bf = [](const uint16_t* p, int e) { return __uint_as_float(uint32_t(p[e]) << 16); };
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf(a.q + i * a.q_ts + h * a.q_hs, lane * E + e);
        acc[e] = 0.f;
    }
    float m = -__builtin_huge_valf(), l = 0.f;
    for (int j = a.cu[lo]; j <= i; ++j) {
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            x = fmaf(q[e], bf(a.k + j * a.k_ts + hk * a.k_hs, lane * E + e), x);
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
        x *= a.scale_log2;
        const float mn = fmaxf(m, x);
        if (mn == -__builtin_huge_valf()) continue;
        const float al = exp2f(m - mn), p = exp2f(x - mn);
        l = l * al + p;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = acc[e] * al + p * bf(a.v + j * a.v_ts + hk * a.v_hs, lane * E + e);
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const __nv_bfloat16 o = __float2bfloat16_rn(acc[e] / l);
        a.out[w * D + lane * E + e] = *reinterpret_cast<const uint16_t*>(&o);
    }
    if (lane == 0) a.lse[w] = (m + log2f(l)) * 0.69314718055994530942f;
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
        (d != 64 && d != 128) || !std::isfinite(softmax_scale))
        return TREE_ATTN_ERR_SHAPE;
    if (B == 0 || N == 0) return TREE_ATTN_OK;
    if (!q || !k || !v || !cu_seqlens || !out || !lse) return TREE_ATTN_ERR_NULL;
    if (!ptr_aligned(q, 16) || !ptr_aligned(k, 16) || !ptr_aligned(v, 16) ||
        !ptr_aligned(out, 16) || !ptr_aligned(lse, 4) || !ptr_aligned(cu_seqlens, 4) ||
        !ptr_aligned(status, 4) || q_token_stride % 8 != 0 || q_head_stride % 8 != 0 ||
        k_token_stride % 8 != 0 || k_head_stride % 8 != 0 || v_token_stride % 8 != 0 ||
        v_head_stride % 8 != 0)
        return TREE_ATTN_ERR_ALIGN;
    PrefillArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.cu = cu_seqlens;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
    const long long rows = static_cast<long long>(N) * Hq;
    if ((rows + 3) / 4 > 0x7fffffffLL) return TREE_ATTN_ERR_SHAPE;
    const cudaError_t e =
        launch_dependent(d == 128 ? prefill_rows_kernel<128> : prefill_rows_kernel<64>,
                         dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
                         static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? TREE_ATTN_OK : TREE_ATTN_ERR_CUDA;
}
