// Causal attention over packed prompts.  C ABI: include/maple_attn.h.
#include <math.h>
#include <stdint.h>

#include "../../include/maple_attn.h"
#include "kv_cache.cuh"

using namespace maple;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// One warp per query row and head, one key at a time with a running maximum
// and sum.
template <typename T, int D>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const maple_attn_prompt_args a)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z, kvh = h / (a.heads / a.kv_heads);
    const int64_t q0 = min(max((int64_t)a.cu_q[b], (int64_t)0), a.Tq), q1 = min(max((int64_t)a.cu_q[b + 1], q0), a.Tq);
    const int64_t k0 = min(max((int64_t)a.cu_k[b], (int64_t)0), a.Tk), k1 = min(max((int64_t)a.cu_k[b + 1], k0), a.Tk);
    if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0 &&
        (a.cu_q[b] != q0 || a.cu_q[b + 1] != q1 || a.cu_k[b] != k0 || a.cu_k[b + 1] != k1 || q1 - q0 > a.max_q))
        set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
    const int64_t i = blockIdx.x * 4ll + (threadIdx.x >> 5);
    if (i >= q1 - q0 || i >= a.max_q) return;
    const int64_t pos = i + (k1 - k0) - (q1 - q0);
    const int64_t first = a.window ? max(pos - a.window + 1, (int64_t)0) : 0;
    float q[E], o[E], mx = -INFINITY, sum = 0.0f;
    const T *qp = (const T *)a.q + (q0 + i) * a.q_stride + (int64_t)h * D + lane * E;
    for (int e = 0; e < E; e++) {
        q[e] = (float)qp[e] * a.scale;
        o[e] = 0.0f;
    }
    for (int64_t j = first; j <= pos; j++) {
        const T *kp = (const T *)a.k + (k0 + j) * a.k_stride + (int64_t)kvh * D + lane * E;
        const T *vp = (const T *)a.v + (k0 + j) * a.v_stride + (int64_t)kvh * D + lane * E;
        float s = 0.0f;
        for (int e = 0; e < E; e++) s = fmaf(q[e], (float)kp[e], s);
        s = warp_tree_sum(s);
        const float m2 = fmaxf(mx, s), c = mx == -INFINITY ? 0.0f : expf(mx - m2), p = expf(s - m2);
        sum = fmaf(sum, c, p);
        for (int e = 0; e < E; e++) o[e] = fmaf(o[e], c, p * (float)vp[e]);
        mx = m2;
    }
    T *op = (T *)a.out + ((q0 + i) * a.heads + h) * D + lane * E;
    for (int e = 0; e < E; e++) op[e] = (T)(pos >= first ? o[e] / sum : 0.0f);
    if (a.lse && lane == 0) a.lse[(q0 + i) * a.heads + h] = pos >= first ? mx + logf(sum) : -INFINITY;
}

}  // namespace

extern "C" int maple_attn_prompt(const maple_attn_prompt_args *args, maple_stream_t stream)
{
    if (!args) return MAPLE_ERR_INVALID_ARG;
    const maple_attn_prompt_args &a = *args;
    const int D = a.head_dim;
    if ((D != 64 && D != 128) || a.heads < 1 || a.kv_heads < 1 || a.heads > 1024 || a.heads % a.kv_heads ||
        a.heads / a.kv_heads > 64)
        return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (a.dtype != MAPLE_BF16 && a.dtype != MAPLE_FP16) return MAPLE_ERR_INVALID_ARG;
    if (a.B < 0 || a.B > 65535 || a.max_q < 0 || a.window < 0 || a.Tq < 0 || a.Tk < 0 || a.Tq > 0x7fffffffll ||
        a.Tk > 0x7fffffffll || !isfinite(a.scale))
        return MAPLE_ERR_INVALID_ARG;
    if (a.B == 0 || a.Tq == 0 || a.max_q == 0) return MAPLE_OK;
    if (!a.q || !a.out || !a.cu_q || !a.cu_k || (a.Tk && (!a.k || !a.v))) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {a.q, a.k, a.v, (const void *)a.out})
        if (!aligned16(p)) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {(const void *)a.cu_q, (const void *)a.cu_k, (const void *)a.lse})
        if ((uintptr_t)p & 3u) return MAPLE_ERR_INVALID_ARG;
    if (a.q_stride % 8 || a.k_stride % 8 || a.v_stride % 8) return MAPLE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid((a.max_q + 3) / 4, a.heads, a.B);
    if (a.dtype == MAPLE_BF16) {
        if (D == 128) prompt_rows_kernel<__nv_bfloat16, 128><<<grid, 128, 0, st>>>(a);
        else prompt_rows_kernel<__nv_bfloat16, 64><<<grid, 128, 0, st>>>(a);
    } else {
        if (D == 128) prompt_rows_kernel<__half, 128><<<grid, 128, 0, st>>>(a);
        else prompt_rows_kernel<__half, 64><<<grid, 128, 0, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}
