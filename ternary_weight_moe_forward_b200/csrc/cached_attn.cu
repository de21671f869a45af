// Attention of one new token per sequence over the paged 4-bit cache.  C ABI:
// include/maple_attn.h.
#include <math.h>
#include <stdint.h>

#include "../../include/maple_attn.h"
#include "kv_cache.cuh"

using namespace maple;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// One warp per sequence and query head, one cached token at a time.
template <typename T, int D>
__global__ void __launch_bounds__(32) cached_rows_kernel(const maple_attn_cached_args a)
{
    using P = KvPage<D>;
    constexpr int E = D / 32;
    const int lane = threadIdx.x, h = blockIdx.x, b = blockIdx.y, kvh = h / (a.heads / a.kv_heads), n = a.page_size;
    int64_t len = a.lens[b];
    if (len > (int64_t)a.max_pages * n) {
        len = (int64_t)a.max_pages * n;
        if (lane == 0) set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
    }
    float q[E], o[E], mx = -INFINITY, sum = 0.0f;
    const T *qp = (const T *)a.q + b * a.q_stride + (int64_t)h * D + lane * E;
    for (int e = 0; e < E; e++) {
        q[e] = (float)qp[e] * a.scale;
        o[e] = 0.0f;
    }
    for (int64_t j = a.window ? max(len - a.window, (int64_t)0) : 0; j < len; j++) {
        const int64_t pg = a.block_table[b * a.table_stride + j / n];
        if (pg < 0 || pg >= a.num_pages) {
            if (lane == 0) set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
            continue;
        }
        const int p = (int)(j % n);
        const uint8_t *base = a.pages + (pg * a.kv_heads + kvh) * P::bytes(n);
        float s = 0.0f, v[E];
        for (int e = 0; e < E; e++) {
            const int c = lane * E + e, w = c / 8, sh = 4 * (c % 8), g = c / 32;
            const uint32_t kw = *(const uint32_t *)(base + P::k_word(p, w)), vw = *(const uint32_t *)(base + P::v_word(n, p, w));
            const float2 kp = __half22float2(*(const __half2 *)(base + P::k_pair(n, p, g)));
            s = fmaf(q[e], fmaf(kp.x, (float)((kw >> sh) & 15u), kp.y), s);
            v[e] = fmaf(__half2float(*(const __half *)(base + P::v_scale(n, p, g))), (float)((vw >> sh) & 15u),
                        __half2float(*(const __half *)(base + P::v_min(n, p, g))));
        }
        s = warp_tree_sum(s);
        const float m2 = fmaxf(mx, s), c = mx == -INFINITY ? 0.0f : expf(mx - m2), pr = expf(s - m2);
        sum = fmaf(sum, c, pr);
        for (int e = 0; e < E; e++) o[e] = fmaf(o[e], c, pr * v[e]);
        mx = m2;
    }
    T *op = (T *)a.out + ((int64_t)b * a.heads + h) * D + lane * E;
    for (int e = 0; e < E; e++) op[e] = (T)(mx == -INFINITY ? 0.0f : o[e] / sum);
}

}  // namespace

extern "C" int64_t maple_attn_cached_workspace(int32_t B, int32_t max_pages, int32_t heads, int32_t kv_heads,
                                               int32_t head_dim, int32_t page_size, int32_t window)
{
    if (maple_attn_page_bytes(head_dim, page_size) < 0 || heads < 1 || kv_heads < 1 || heads > 1024 || heads % kv_heads)
        return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (B < 0 || B > 65535 || max_pages < 0 || window < 0) return MAPLE_ERR_INVALID_ARG;
    return 0;
}

extern "C" int maple_attn_cached(const maple_attn_cached_args *args, maple_stream_t stream)
{
    if (!args) return MAPLE_ERR_INVALID_ARG;
    const maple_attn_cached_args &a = *args;
    const int64_t need = maple_attn_cached_workspace(a.B, a.max_pages, a.heads, a.kv_heads, a.head_dim, a.page_size, a.window);
    if (need < 0) return (int)need;
    if (a.dtype != MAPLE_BF16 && a.dtype != MAPLE_FP16) return MAPLE_ERR_INVALID_ARG;
    if (!isfinite(a.scale)) return MAPLE_ERR_INVALID_ARG;
    if (a.B == 0) return MAPLE_OK;
    if (!a.q || !a.out || !a.lens || (a.max_pages && (!a.pages || !a.block_table || a.num_pages < 1)) ||
        a.num_pages > (1ll << 40))
        return MAPLE_ERR_INVALID_ARG;
    if (need && (!a.workspace || a.workspace_bytes < need)) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {a.q, (const void *)a.out, (const void *)a.pages, (const void *)a.workspace})
        if (!aligned16(p)) return MAPLE_ERR_INVALID_ARG;
    if (((uintptr_t)a.block_table & 3u) || ((uintptr_t)a.lens & 3u) || a.q_stride % 8) return MAPLE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid(a.heads, a.B);
    if (a.dtype == MAPLE_BF16) {
        if (a.head_dim == 128) cached_rows_kernel<__nv_bfloat16, 128><<<grid, 32, 0, st>>>(a);
        else cached_rows_kernel<__nv_bfloat16, 64><<<grid, 32, 0, st>>>(a);
    } else {
        if (a.head_dim == 128) cached_rows_kernel<__half, 128><<<grid, 32, 0, st>>>(a);
        else cached_rows_kernel<__half, 64><<<grid, 32, 0, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}
