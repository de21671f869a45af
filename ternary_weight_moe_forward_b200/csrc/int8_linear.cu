// Int8 linear layer: rows quantised to int8 (absmax, one scale per token),
// times int8 weights with one scale per output channel.  C ABI:
// include/maple_attn.h.
#include <stdint.h>

#include "../../include/maple_attn.h"
#include <cuda_bf16.h>

#include "common.cuh"

using namespace maple;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Int8 absmax codes of bf16 rows, one warp per row; the second pass over the
// row hits L1 or L2.
__global__ void __launch_bounds__(256) quantise_rows_kernel(const uint16_t *x, int64_t stride, int64_t T, int K, int8_t *q,
                                                            float *s)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (t >= T) return;
    const uint4 *xr = reinterpret_cast<const uint4 *>(x + t * stride);
    float amax = 0.0f;
    for (int c = lane; c < K / 8; c += 32) {
        const uint4 v = __ldg(xr + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int m = 0; m < 4; m++) {
            amax = fmaxf(amax, fabsf(bf16_bits_to_f32(w[m] & 0xffffu)));
            amax = fmaxf(amax, fabsf(bf16_bits_to_f32(w[m] >> 16)));
        }
    }
    amax = warp_max(amax);
    const float inv = amax > 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
    for (int c = lane; c < K / 8; c += 32) {
        const uint4 v = __ldg(xr + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t pk[2] = {0u, 0u};
#pragma unroll
        for (int m = 0; m < 8; m++) {
            const uint32_t bits = (m & 1) ? (w[m >> 1] >> 16) : (w[m >> 1] & 0xffffu);
            const int code = amax > 0.0f ? quant_code(bf16_bits_to_f32(bits), inv) : 0;
            pk[m >> 2] |= (uint32_t)(code & 0xff) << (8 * (m & 3));
        }
        reinterpret_cast<uint2 *>(q + t * K)[c] = make_uint2(pk[0], pk[1]);
    }
    if (lane == 0) s[t] = amax > 0.0f ? __fdiv_rn(amax, 127.0f) : 0.0f;
}

// One warp per row: bf16(RMSNorm(row)) in shared memory, then its codes
__global__ void __launch_bounds__(128) norm_quantise_rows_kernel(const float *x, int64_t stride, int64_t T, int K,
                                                                 int8_t *q, float *s)
{
    extern __shared__ __align__(16) uint16_t rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x * (int64_t)(blockDim.x >> 5) + warp;
    if (t >= T) return;
    uint16_t *row = rows + (size_t)warp * K;
    rmsnorm_token_warp(x + t * stride, K, row);
    __syncwarp();
    float amax = 0.0f;
    for (int c = lane; c < K / 2; c += 32) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(row)[c];
        amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_f32(w & 0xffffu)), fabsf(bf16_bits_to_f32(w >> 16))));
    }
    amax = warp_max(amax);
    const float inv = amax > 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
    for (int c = lane; c < K / 4; c += 32) {
        const uint2 w = reinterpret_cast<const uint2 *>(row)[c];
        uint32_t pk = 0;
#pragma unroll
        for (int m = 0; m < 4; m++) {
            const uint32_t word = m < 2 ? w.x : w.y, bits = (m & 1) ? word >> 16 : word & 0xffffu;
            const int code = amax > 0.0f ? quant_code(bf16_bits_to_f32(bits), inv) : 0;
            pk |= (uint32_t)(code & 0xff) << (8 * m);
        }
        reinterpret_cast<uint32_t *>(q + t * K)[c] = pk;
    }
    if (lane == 0) s[t] = amax > 0.0f ? __fdiv_rn(amax, 127.0f) : 0.0f;
}

struct LinearOut {
    const float *alpha, *bias, *resid;
    void *y;
    int64_t N;
    int y_bf16;
    __device__ __forceinline__ void store(int64_t t, int64_t n, int acc, float s) const
    {
        float v = __fmul_rn((float)acc, __fmul_rn(alpha[n], s));
        if (bias) v = __fadd_rn(v, bias[n]);
        if (resid) v = __fadd_rn(resid[t * N + n], v);
        if (y_bf16) ((uint16_t *)y)[t * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        else ((float *)y)[t * N + n] = v;
    }
};

// One thread per output
__global__ void __launch_bounds__(256) linear_dp4a_kernel(const int8_t *q, const float *s, const int8_t *w, int64_t T, int K,
                                                          LinearOut o)
{
    const int64_t n = blockIdx.x * 32ll + (threadIdx.x & 31), t = blockIdx.y * 8ll + (threadIdx.x >> 5);
    if (n >= o.N || t >= T) return;
    const uint4 *a = reinterpret_cast<const uint4 *>(q + t * K), *b = reinterpret_cast<const uint4 *>(w + n * K);
    int acc = 0;
    for (int c = 0; c < K / 16; c++) {
        const uint4 u = a[c], v = b[c];
        acc = __dp4a((int)u.x, (int)v.x, acc);
        acc = __dp4a((int)u.y, (int)v.y, acc);
        acc = __dp4a((int)u.z, (int)v.z, acc);
        acc = __dp4a((int)u.w, (int)v.w, acc);
    }
    o.store(t, n, acc, s[t]);
}

int64_t round256(int64_t v) { return (v + 255) & ~255ll; }

int check_sizes(int64_t T, int64_t K, int64_t N)
{
    if (K < 16 || K > 32768 || K % 16 || N < 1) return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (T < 0 || T >= 0x7fffffffll || N >= 0x7fffffffll || T * N >= (1ll << 40) || N * K >= (1ll << 40))
        return MAPLE_ERR_UNSUPPORTED_SHAPE;
    return MAPLE_OK;
}

}  // namespace

extern "C" int64_t maple_attn_linear_workspace(int64_t T, int64_t K, int64_t N)
{
    const int rc = check_sizes(T, K, N);
    if (rc) return rc;
    return round256(T * K) + round256(T * 4);
}

extern "C" int maple_attn_linear(const maple_attn_linear_args *args, maple_stream_t stream)
{
    if (!args) return MAPLE_ERR_INVALID_ARG;
    const maple_attn_linear_args &a = *args;
    const int64_t need = maple_attn_linear_workspace(a.T, a.K, a.N);
    if (need < 0) return (int)need;
    if (a.normalise && a.K % 256) return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (a.y_dtype != MAPLE_BF16 && a.y_dtype != MAPLE_FP32) return MAPLE_ERR_INVALID_ARG;
    if (a.T == 0) return MAPLE_OK;
    if (!a.x || !a.w || !a.alpha || !a.y || !a.workspace || a.workspace_bytes < need) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {a.x, (const void *)a.w, (const void *)a.alpha, (const void *)a.bias, (const void *)a.resid,
                          (const void *)a.y, (const void *)a.workspace})
        if (!aligned16(p)) return MAPLE_ERR_INVALID_ARG;
    if (a.x_stride % 8) return MAPLE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    int8_t *q = (int8_t *)a.workspace;
    float *s = (float *)((char *)a.workspace + round256(a.T * a.K));
    const int K = (int)a.K;
    if (a.normalise) {
        const int warps = K <= 4096 ? 4 : 1;   // (K bf16 values of shared memory a warp: 32 KB at most below the opt-in limit)
        if ((size_t)warps * K * 2 > 49152 &&
            cudaFuncSetAttribute(norm_quantise_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536) != cudaSuccess) {
            cudaGetLastError();
            return MAPLE_ERR_CUDA;
        }
        norm_quantise_rows_kernel<<<(unsigned)((a.T + warps - 1) / warps), warps * 32, (size_t)warps * K * 2, st>>>(
            (const float *)a.x, a.x_stride, a.T, K, q, s);
    } else {
        quantise_rows_kernel<<<(unsigned)((a.T + 7) / 8), 256, 0, st>>>((const uint16_t *)a.x, a.x_stride, a.T, K, q, s);
    }
    const LinearOut o{a.alpha, a.bias, a.resid, a.y, a.N, a.y_dtype == MAPLE_BF16};
    if ((a.T + 7) / 8 > 65535) return MAPLE_ERR_UNSUPPORTED_SHAPE;
    linear_dp4a_kernel<<<dim3((unsigned)((a.N + 31) / 32), (unsigned)((a.T + 7) / 8)), 256, 0, st>>>(q, s, a.w, a.T, K, o);
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}
