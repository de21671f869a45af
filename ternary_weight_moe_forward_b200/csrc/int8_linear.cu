// Int8 linear layer: rows quantised to int8 (absmax, one scale per token),
// times int8 weights with one scale per output channel.  C ABI:
// include/maple_attn.h.
//
// The sums are integers (exact), so nothing depends on how K is cut or ordered,
// and every path gives the same bits.  Two paths, by the number of tokens:
//   T <= 16   linear_rows_kernel: the weights are streamed once through
//             warp-level int8 matrix instructions by all SMs, the tokens are
//             quantised (normed first, for at most 16384 values) in the same
//             kernel;
//   others    quantise_rows_kernel or norm_quantise_rows_kernel, then
//             linear_gemm_kernel on tcgen05 (kind::i8).  Up to 128 tokens the
//             weights are the 128-row operand and all tokens one N tile (the
//             weights are read once); above, the tokens are.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/maple_attn.h"
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

using namespace maple;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// The largest absolute value of a row, or NaN if the row holds one: its codes mean
// nothing then, and a scale of NaN makes the row's outputs NaN.  (An infinity does
// the same without help: scale infinite, all codes 0.)
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(FULL, v, o));
    return v;
}
__device__ __forceinline__ float row_inv(float amax) { return amax > 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f; }   // (a zero row: codes 0)
__device__ __forceinline__ float row_scale(float amax) { return amax > 0.0f ? __fdiv_rn(amax, 127.0f) : amax; }

// Int8 absmax codes of bf16 rows, one warp per row.  NV > 0: the row (at most
// 256 NV values) stays in registers between the maximum and the codes, all of
// its loads in flight; NV = 0: longer rows are read twice, the second time from
// L1 or L2.
__device__ __forceinline__ uint2 quant8(const uint4 &v, float inv)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t pk[2] = {0u, 0u};
#pragma unroll
    for (int m = 0; m < 8; m++) {
        const uint32_t bits = (m & 1) ? (w[m >> 1] >> 16) : (w[m >> 1] & 0xffffu);
        pk[m >> 2] |= (uint32_t)(quant_code(bf16_bits_to_f32(bits), inv) & 0xff) << (8 * (m & 3));
    }
    return make_uint2(pk[0], pk[1]);
}
__device__ __forceinline__ float absmax8(const uint4 &v, float amax)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int m = 0; m < 4; m++)
        amax = max_nan(amax, max_nan(fabsf(bf16_bits_to_f32(w[m] & 0xffffu)), fabsf(bf16_bits_to_f32(w[m] >> 16))));
    return amax;
}

template <int NV>
__global__ void __launch_bounds__(256) quantise_rows_kernel(const uint16_t *x, int64_t stride, int64_t T, int K, int8_t *q,
                                                            float *s)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x * 8ll + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.launch_dependents;");
    if (t >= T) return;
    const uint4 *xr = reinterpret_cast<const uint4 *>(x + t * stride);
    uint2 *qr = reinterpret_cast<uint2 *>(q + t * K);
    const int n = K / 8;
    uint4 v[NV > 0 ? NV : 1];
    float amax = 0.0f;
    if (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; i++) v[i] = lane + 32 * i < n ? __ldg(xr + lane + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < NV; i++) amax = absmax8(v[i], amax);
    } else {
        for (int c = lane; c < n; c += 32) amax = absmax8(__ldg(xr + c), amax);
    }
    amax = warp_max_nan(amax);
    const float inv = row_inv(amax);
    if (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (lane + 32 * i < n) qr[lane + 32 * i] = quant8(v[i], inv);
    } else {
        for (int c = lane; c < n; c += 32) qr[c] = quant8(__ldg(xr + c), inv);
    }
    if (lane == 0) s[t] = row_scale(amax);
}

// Sum of the squares of a row, one warp, in the order of rmsnorm_token_warp
__device__ __forceinline__ float sum_squares_warp(const float *r, int K)
{
    const int lane = threadIdx.x & 31;
    float acc = 0.0f;
    for (int i = 0; i < K / 256; i++) {
        const float4 v0 = *reinterpret_cast<const float4 *>(r + 256 * i + 8 * lane);
        const float4 v1 = *reinterpret_cast<const float4 *>(r + 256 * i + 8 * lane + 4);
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int m = 0; m < 8; m++) acc = __fmaf_rn(v[m], v[m], acc);
    }
    return warp_tree_sum(acc);
}

// One warp per row: bf16(RMSNorm(row)) in shared memory, then its codes.  A row
// whose sum of squares is not finite has no norm: its normed values come out as
// zeros (so only rows of zeros are looked at again), its scale has to be NaN.
__global__ void __launch_bounds__(128) norm_quantise_rows_kernel(const float *x, int64_t stride, int64_t T, int K,
                                                                 int8_t *q, float *s)
{
    extern __shared__ __align__(16) uint16_t rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x * (int64_t)(blockDim.x >> 5) + warp;
    asm volatile("griddepcontrol.launch_dependents;");
    if (t >= T) return;
    uint16_t *row = rows + (size_t)warp * K;
    rmsnorm_token_warp(x + t * stride, K, row);
    __syncwarp();
    float amax = 0.0f;
    for (int c = lane; c < K / 2; c += 32) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(row)[c];
        amax = max_nan(amax, max_nan(fabsf(bf16_bits_to_f32(w & 0xffffu)), fabsf(bf16_bits_to_f32(w >> 16))));
    }
    amax = warp_max_nan(amax);
    const float inv = row_inv(amax);
    if (!(amax > 0.0f) && !(sum_squares_warp(x + t * stride, K) < INFINITY)) amax = NAN;
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
    if (lane == 0) s[t] = row_scale(amax);
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

// ---------------------------------------------------------------------------
// T <= 16.  A CTA takes 16 output channels at a time (m16n8k32, the weights as
// the 16-row operand, tokens as columns), its 16 warps sharing K in pieces of 64
// bytes: lane (g, t) reads 16 contiguous bytes of rows g and g + 8, and since the
// order of the sum does not matter these are its fragments of two instructions,
// against the same 16 bytes of token g's codes.  The weights go from memory to
// registers in 16-byte loads, the next channels' before this one's sums are
// joined.  Bound by HBM for a large N, by latency for one projection.
// ---------------------------------------------------------------------------
constexpr int kRowWarps = 16, kRowUnits = 2;   // warps of a CTA; 64-byte pieces of K in flight per warp

__host__ __device__ __forceinline__ int row_pitch(int K)   // bytes of a token's codes: an odd multiple of 64 (no bank conflicts)
{
    const int u = (K + 63) / 64;
    return 64 * (u | 1);
}

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes of bf16(RMSNorm(r)) of one fp32 row, one warp: the steps of
// rmsnorm_token_warp (the same order of the sum, the same roundings) with the
// normed row computed again for its maximum and for its codes instead of kept.
__device__ __forceinline__ void norm_codes_warp(const float *r, int K, uint8_t *row, float *scale)
{
    const int lane = threadIdx.x & 31;
    const float rms = __fsqrt_rn(__fadd_rn(__fdiv_rn(sum_squares_warp(r, K), (float)K), 1e-6f));
    auto normed = [&](int i) -> uint4 {
        const float4 v0 = *reinterpret_cast<const float4 *>(r + 256 * i + 8 * lane);
        const float4 v1 = *reinterpret_cast<const float4 *>(r + 256 * i + 8 * lane + 4);
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t pk[4];
#pragma unroll
        for (int m = 0; m < 4; m++)
            pk[m] = (uint32_t)f32_to_bf16_bits(__fdiv_rn(v[2 * m], rms)) | ((uint32_t)f32_to_bf16_bits(__fdiv_rn(v[2 * m + 1], rms)) << 16);
        return make_uint4(pk[0], pk[1], pk[2], pk[3]);
    };
    float amax = 0.0f;
    for (int i = 0; i < K / 256; i++) amax = absmax8(normed(i), amax);
    amax = warp_max(amax);
    const float inv = row_inv(amax);
    for (int i = 0; i < K / 256; i++) reinterpret_cast<uint2 *>(row)[32 * i + lane] = quant8(normed(i), inv);
    if (lane == 0) *scale = rms < INFINITY ? row_scale(amax) : NAN;   // (a sum of squares that is not finite: no norm)
}

// NT: column tiles of 8 tokens; NORM: x is the fp32 residual stream
template <int NT, bool NORM>
__global__ void __launch_bounds__(kRowWarps * 32, 2)
linear_rows_kernel(const void *xv, int64_t x_stride, int T, int K, const int8_t *w, LinearOut o)
{
    const uint16_t *x = (const uint16_t *)xv;
    extern __shared__ __align__(16) uint8_t codes[];        // [8 NT][pitch], then [2][16 warps][NT][32 lanes] int4
    __shared__ float s_scale[8 * NT], s_part[kRowWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int pitch = row_pitch(K), units = (K + 63) / 64;
    int4 *red = (int4 *)(codes + 8 * NT * pitch);
    const int64_t tiles = (o.N + 15) / 16;

    uint4 wa[kRowUnits], wb[kRowUnits];
    auto fetch = [&](int64_t tile, int u0) {      // the warp's pieces u0, u0 + 16, ... of a tile's rows
#pragma unroll
        for (int i = 0; i < kRowUnits; i++) {
            const int64_t r = tile * 16 + g;
            const int k = 64 * (u0 + kRowWarps * i) + 16 * t;
            const bool in = k < K;
            wa[i] = in && r < o.N ? ld_stream_v4(w + r * K + k) : make_uint4(0, 0, 0, 0);
            wb[i] = in && r + 8 < o.N ? ld_stream_v4(w + (r + 8) * K + k) : make_uint4(0, 0, 0, 0);
        }
    };
    if ((int64_t)blockIdx.x < tiles) fetch(blockIdx.x, warp);   // in flight while the tokens are quantised

    // ---- the tokens' codes, two per round (eight warps each); rows beyond T are 0
    if (NORM && warp < 8 * NT) {   // a warp per token (16 warps, at most 16 tokens)
        uint8_t *row = codes + warp * pitch;
        if (warp < T) norm_codes_warp((const float *)xv + warp * x_stride, K, row, s_scale + warp);
        for (int c = (warp < T ? K : 0) / 16 + lane; c < pitch / 16; c += 32) reinterpret_cast<uint4 *>(row)[c] = make_uint4(0, 0, 0, 0);
    }
    for (int r0 = 0; !NORM && r0 < 8 * NT; r0 += 2) {
        const int r = r0 + (warp >> 3), tid = threadIdx.x & 255;
        uint8_t *row = codes + r * pitch;
        if (r0 >= T) {   // (T is the same for all threads)
            for (int c = tid; c < pitch / 16; c += 256) reinterpret_cast<uint4 *>(row)[c] = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint4 *xr = reinterpret_cast<const uint4 *>(x + (int64_t)min(r, T - 1) * x_stride);
        float amax = 0.0f;
        for (int c = tid; c < K / 8; c += 256) {
            const uint4 v = __ldg(xr + c);
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int m = 0; m < 4; m++)
                amax = max_nan(amax, max_nan(fabsf(bf16_bits_to_f32(q[m] & 0xffffu)), fabsf(bf16_bits_to_f32(q[m] >> 16))));
        }
        amax = warp_max_nan(amax);
        __syncthreads();
        if (lane == 0) s_part[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; i++) amax = max_nan(amax, s_part[(warp & 8) + i]);
        if (r >= T) amax = 0.0f;
        const float inv = row_inv(amax);
        for (int c = tid; c < pitch / 8; c += 256) {
            uint32_t pk[2] = {0u, 0u};
            if (c < K / 8 && amax > 0.0f) {
                const uint4 v = __ldg(xr + c);
                const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int m = 0; m < 8; m++) {
                    const uint32_t bits = (m & 1) ? (q[m >> 1] >> 16) : (q[m >> 1] & 0xffffu);
                    pk[m >> 2] |= (uint32_t)(quant_code(bf16_bits_to_f32(bits), inv) & 0xff) << (8 * (m & 3));
                }
            }
            reinterpret_cast<uint2 *>(row)[c] = make_uint2(pk[0], pk[1]);
        }
        if (tid == 0) s_scale[r] = row_scale(amax);
    }
    __syncthreads();

    int buf = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
        int c[NT][4];
#pragma unroll
        for (int j = 0; j < NT; j++) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0;
        for (int u0 = warp; u0 < units; u0 += kRowWarps * kRowUnits) {
            uint4 a[kRowUnits], b[kRowUnits];
#pragma unroll
            for (int i = 0; i < kRowUnits; i++) {
                a[i] = wa[i];
                b[i] = wb[i];
            }
            // the next pieces: of this tile, or the first of the CTA's next tile
            const int next = u0 + kRowWarps * kRowUnits;
            if (next < units) fetch(tile, next);
            else if (tile + gridDim.x < tiles) fetch(tile + gridDim.x, warp);
#pragma unroll
            for (int i = 0; i < kRowUnits; i++) {
                const int u = u0 + kRowWarps * i;
                if (u >= units) break;
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(codes + (8 * j + g) * pitch + 64 * u + 16 * t);
                    mma_s8(c[j], a[i].x, b[i].x, a[i].y, b[i].y, q.x, q.y);
                    mma_s8(c[j], a[i].z, b[i].z, a[i].w, b[i].w, q.z, q.w);
                }
            }
        }
        if (warp >= units && tile + gridDim.x < tiles) fetch(tile + gridDim.x, warp);   // (a warp without a piece of K: zeros)
#pragma unroll
        for (int j = 0; j < NT; j++)
            red[((buf * kRowWarps + warp) * NT + j) * 32 + lane] = make_int4(c[j][0], c[j][1], c[j][2], c[j][3]);
        __syncthreads();
        // output (token, channel): lane 4 (channel % 8) + token % 8 / 2, word 2 (channel / 8) + token % 2
        for (int i = threadIdx.x; i < 16 * T; i += kRowWarps * 32) {
            const int tok = i >> 4, ch = i & 15;
            const int *src = (const int *)red + (((buf * kRowWarps) * NT + (tok >> 3)) * 32 + 4 * (ch & 7) + ((tok & 7) >> 1)) * 4 +
                             2 * (ch >> 3) + (tok & 1);
            int acc = 0;
#pragma unroll
            for (int v = 0; v < kRowWarps; v++) acc += src[v * NT * 128];
            if (tile * 16 + ch < o.N) o.store(tok, tile * 16 + ch, acc, s_scale[tok]);
        }
    }
}

// ---------------------------------------------------------------------------
// T > 16.  D[128 rows of A][bn rows of B], both operands K-major int8 tiles of
// 128 bytes of K by TMA with the 128-byte swizzle, int32 accumulators in tensor
// memory, two of them, so that the epilogue of a tile runs under the next one's
// products.  SWAP: A is the weights and B the tokens (T <= 128), else the other
// way round.  Warp 0 loads, warp 1 issues the products, warps 4-11 scale and
// store.  CTAs take tiles round robin.
// ---------------------------------------------------------------------------
constexpr int kGemmThreads = 384, kGemmBK = 128;

struct GemmArgs {
    LinearOut o;
    const float *s;
    int64_t T;
    int K, bn, stages;
    int64_t tiles_a, tiles_b;
    int y_tma;                 // y is written by TMA (its rows are multiples of 16 bytes)
    unsigned *flag;
};

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mma_i8_plain(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

// four values from index i on, 0 beyond n
__device__ __forceinline__ float4 load4(const float *p, int64_t i, int64_t n)
{
    if (i + 4 <= n) return *reinterpret_cast<const float4 *>(p + i);
    return make_float4(i < n ? p[i] : 0.0f, i + 1 < n ? p[i + 1] : 0.0f, i + 2 < n ? p[i + 2] : 0.0f, 0.0f);
}

template <bool SWAP>
__global__ void __launch_bounds__(kGemmThreads, 1)
linear_gemm_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                   const __grid_constant__ CUtensorMap y_map, const GemmArgs p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    // (a broadcast index: the products' operands stay in uniform registers)
    const int warp = __shfl_sync(FULL, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (smem_addr(smem) & 1023u) {   // the swizzled tiles need 1024-byte alignment
        if (threadIdx.x == 0) set_flag(p.flag, MAPLE_DEVFLAG_TIMEOUT);
        return;
    }
    const int S = p.stages, bn = p.bn;
    const uint32_t stage_bytes = (128 + bn) * kGemmBK;
    uint8_t *s_out = smem + S * stage_bytes;                       // [8 epilogue warps][4 KB] rows on their way to y
    float *s_cols = (float *)(s_out + (SWAP ? 0 : 8 * 4096));      // [8 warps][alpha, bias][128]: the warp's columns of a tile
    uint64_t *bars = (uint64_t *)((uint8_t *)s_cols + (SWAP ? 0 : 8 * 1024));
    const uint32_t b_full = smem_addr(bars), b_empty = b_full + 8 * S, b_acc = b_empty + 8 * S, b_free = b_acc + 16, b_drain = b_free + 16;
    uint32_t *tmem_holder = (uint32_t *)(bars + 2 * S + 5);
    volatile uint32_t *abort = tmem_holder + 1;
    const uint64_t limit = kDefaultWaitNs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; i++) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(b_acc + 8 * i, 1);
            mbar_init(b_free + 8 * i, 8);
        }
        mbar_init(b_drain, 1);
        *abort = 0u;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(smem_addr(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int KS = (p.K + kGemmBK - 1) / kGemmBK;      // (columns beyond K arrive as zeros)
    const int64_t tiles = p.tiles_a * p.tiles_b;

    if (warp == 0) {
        // ---------------- loads
        if (lane == 0) {
            uint32_t it = 0, wrap = 0;   // stage, times round
            int s = 0;
            bool ok = true, waited = false;
            for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
                const int64_t ta = tile / p.tiles_b, tb = tile - ta * p.tiles_b;
                for (int k = 0; k < KS; k++, it++) {
                    if (!(ok = mbar_wait(b_empty + 8 * s, (wrap & 1) ^ 1, abort, p.flag, limit))) break;
                    const uint32_t dst = smem_addr(smem) + s * stage_bytes, bar = b_full + 8 * s;
                    mbar_expect_tx(bar, stage_bytes);
                    if (SWAP) {
                        // the weights do not wait for the kernel that quantises the tokens
                        tma_load_2d(dst, &a_map, k * kGemmBK, (int)(ta * 128), bar);
                        if (!waited && (it + 1 == (uint32_t)S || (tile + gridDim.x >= tiles && k + 1 == KS))) {
                            asm volatile("griddepcontrol.wait;" ::: "memory");
                            waited = true;
                            for (int q = 0; q <= s; q++) {   // the token tiles of the stages filled so far
                                const int64_t qt = blockIdx.x + (int64_t)(q / KS) * gridDim.x;
                                tma_load_2d(smem_addr(smem) + q * stage_bytes + 128 * kGemmBK, &b_map, (q % KS) * kGemmBK,
                                            (int)((qt % p.tiles_b) * bn), b_full + 8 * q);
                            }
                        } else if (waited) {
                            tma_load_2d(dst + 128 * kGemmBK, &b_map, k * kGemmBK, (int)(tb * bn), bar);
                        }
                    } else {
                        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
                        waited = true;
                        tma_load_2d(dst, &a_map, k * kGemmBK, (int)(ta * 128), bar);
                        tma_load_2d(dst + 128 * kGemmBK, &b_map, k * kGemmBK, (int)(tb * bn), bar);
                    }
                    if (++s == S) {
                        s = 0;
                        wrap++;
                    }
                }
            }
            if (!ok) {   // drain the copies in flight: each arrives or runs out of time
                for (int q = 0; q < S; q++) {
                    const uint64_t c0 = global_ns();
                    while (global_ns() - c0 < 20000000ull && !(mbar_test(b_full + 8 * q, 0) && mbar_test(b_full + 8 * q, 1))) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- products
        if (elect_one()) {
            const uint32_t idesc = idesc_i8(bn);
            const uint64_t d0 = desc_sw128(smem_addr(smem));
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return mbar_poll(bar, parity) || mbar_wait(bar, parity, abort, p.flag, limit);
            };
            uint32_t wrap = 0, n = 0;
            int s = 0;
            bool ok = true;
            for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x, n++) {
                const uint32_t d = tmem + 256 * (n & 1);
                if (!(ok = wait(b_free + 8 * (n & 1), ((n >> 1) & 1) ^ 1))) break;
                for (int k = 0; k < KS; k++) {
                    if (!(ok = wait(b_full + 8 * s, wrap & 1))) break;
                    tc_fence_after();
                    const uint64_t da = d0 + (uint64_t)(s * (stage_bytes / 16)), db = da + 128 * kGemmBK / 16;
#pragma unroll
                    for (int q = 0; q < kGemmBK / 32; q++) mma_i8_plain(d, da + 2 * q, db + 2 * q, idesc, k > 0 || q > 0);
                    mma_commit(b_empty + 8 * s);
                    if (k + 1 == KS) mma_commit(b_acc + 8 * (n & 1));
                    if (++s == S) {
                        s = 0;
                        wrap++;
                    }
                }
            }
            mma_commit(b_drain);   // every issued MMA has finished before tensor memory is released
            const uint64_t c0 = global_ns();
            while (!mbar_test(b_drain, 0) && global_ns() - c0 < limit) {
            }
        }
    } else if (warp >= 4) {
        // ---------------- epilogue: lane quarter warp % 4, every other 32 columns
        asm volatile("griddepcontrol.wait;" ::: "memory");   // (the scales)
        const int q = warp & 3, half = (warp - 4) >> 2, r = 32 * q + lane;
        const LinearOut &o = p.o;
        uint32_t n = 0, piece = 0;      // tiles, pieces of 32 x 32 outputs that this warp has handed to TMA
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, n++) {
            const int64_t ta = tile / p.tiles_b, tb = tile - ta * p.tiles_b;
            const int64_t row = ta * 128 + r;
            const bool in = row < (SWAP ? o.N : p.T);
            const float fr = in ? (SWAP ? __ldg(o.alpha + row) : __ldg(p.s + row)) : 0.0f;
            float *my_alpha = s_cols + (warp - 4) * 256, *my_bias = my_alpha + 128;
            if (!SWAP) {   // the columns' scales, loaded while the products run
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int64_t c = tb * bn + 32 * half + 64 * i + lane;
                    const bool on = 32 * half + 64 * i < bn && c < o.N;
                    my_alpha[32 * i + lane] = on ? __ldg(o.alpha + c) : 0.0f;
                    my_bias[32 * i + lane] = on && o.bias ? __ldg(o.bias + c) : 0.0f;
                }
                __syncwarp();
            }
            if (!__all_sync(FULL, mbar_wait(b_acc + 8 * (n & 1), (n >> 1) & 1, abort, p.flag, limit))) break;
            tc_fence_after();
            const uint32_t src = tmem + 256 * (n & 1) + ((uint32_t)(32 * q) << 16);
            for (int c0 = 32 * half; c0 < bn; c0 += 64) {
                int acc[32];
                tmem_ld32(src + c0, acc);
                tmem_wait_ld();
                const int64_t col = tb * bn + c0;
                if (SWAP) {
                    // lane = channel, columns = tokens: a warp writes 32 neighbours of a token's row
#pragma unroll
                    for (int c = 0; c < 32; c++)
                        if (in && col + c < p.T) o.store(col + c, row, acc[c], __ldg(p.s + col + c));
                } else {
                    // lane = token, columns = channels
                    float v[32];
                    if (p.y_tma) {
                        // 32 rows x 32 channels through shared memory, so that y is written in whole
                        // row pieces: stored by the lanes (16 bytes of 32 rows at a time), the
                        // epilogue took longer than the products
                        const float4 *al4 = reinterpret_cast<const float4 *>(my_alpha + (c0 >> 6) * 32);
                        const float4 *bi4 = reinterpret_cast<const float4 *>(my_bias + (c0 >> 6) * 32);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 al = al4[c / 4];
                            v[c] = __fmul_rn((float)acc[c], __fmul_rn(al.x, fr));
                            v[c + 1] = __fmul_rn((float)acc[c + 1], __fmul_rn(al.y, fr));
                            v[c + 2] = __fmul_rn((float)acc[c + 2], __fmul_rn(al.z, fr));
                            v[c + 3] = __fmul_rn((float)acc[c + 3], __fmul_rn(al.w, fr));
                        }
                        if (o.bias) {
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 bi = bi4[c / 4];
                                v[c] = __fadd_rn(v[c], bi.x);
                                v[c + 1] = __fadd_rn(v[c + 1], bi.y);
                                v[c + 2] = __fadd_rn(v[c + 2], bi.z);
                                v[c + 3] = __fadd_rn(v[c + 3], bi.w);
                            }
                        }
                        if (o.resid && in) {
#pragma unroll
                            for (int c = 0; c < 32; c += 4) {
                                const float4 re = load4(o.resid + row * o.N, col + c, o.N);
                                v[c] = __fadd_rn(re.x, v[c]);
                                v[c + 1] = __fadd_rn(re.y, v[c + 1]);
                                v[c + 2] = __fadd_rn(re.z, v[c + 2]);
                                v[c + 3] = __fadd_rn(re.w, v[c + 3]);
                            }
                        }
                        // Two pieces of bf16 fit the warp's 4 KB, one of fp32.  The halves alternate from piece to
                        // piece over all tiles of the CTA: the wait below leaves the newest store pending, which
                        // then always reads the other half.  (Counted from each tile's start, the last piece of a
                        // tile with an odd number of them and the next tile's first would share one.)
                        uint8_t *st = s_out + (warp - 4) * 4096 + (o.y_bf16 ? (piece++ & 1) * 2048 : 0);
                        if (lane == 0) {
                            if (o.y_bf16) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                            else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        }
                        __syncwarp();
                        if (o.y_bf16) {      // rows of 64 bytes, 64-byte swizzle
#pragma unroll
                            for (int c = 0; c < 32; c += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int z = 0; z < 4; z++) {
                                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[c + 2 * z], v[c + 2 * z + 1]);
                                    w[z] = *reinterpret_cast<const uint32_t *>(&b);
                                }
                                *reinterpret_cast<uint4 *>(st + lane * 64 + (((c / 8) ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {             // rows of 128 bytes, 128-byte swizzle
#pragma unroll
                            for (int c = 0; c < 32; c += 4)
                                *reinterpret_cast<float4 *>(st + lane * 128 + (((c / 4) ^ (lane & 7)) << 4)) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0 && ta * 128 + 32 * q < p.T && col < o.N) {   // (rows and columns beyond y are cut off)
                            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                                             reinterpret_cast<uint64_t>(&y_map)),
                                         "r"(smem_addr(st)), "r"((int)col), "r"((int)(ta * 128 + 32 * q))
                                         : "memory");
                        }
                        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");   // (an empty one too: they are counted)
                    } else if (in) {
#pragma unroll
                        for (int c = 0; c < 32; c++)
                            if (col + c < o.N) o.store(row, col + c, acc[c], fr);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_free + 8 * (n & 1));
        }
        // (shared memory must outlive the stores that read it)
        if (!SWAP && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

typedef CUresult (*encode_fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

encode_fn encoder()
{
    static encode_fn encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (encode_fn)fn;
    }();
    return encode;
}

// int8 [rows][K], boxes of `box` rows x 128 bytes, 128-byte swizzle
int row_map(CUtensorMap *map, const void *base, int64_t rows, int64_t K, int box)
{
    encode_fn encode = encoder();
    if (!encode) return MAPLE_ERR_CUDA;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K};
    cuuint32_t b[2] = {kGemmBK, (cuuint32_t)box}, estr[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, b, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MAPLE_OK : MAPLE_ERR_CUDA;
}

// y [T][N], boxes of 32 rows x 32 columns
int out_map(CUtensorMap *map, void *y, int64_t T, int64_t N, bool bf16)
{
    encode_fn encode = encoder();
    if (!encode) return MAPLE_ERR_CUDA;
    cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)T};
    cuuint64_t strides[1] = {(cuuint64_t)N * (bf16 ? 2 : 4)};
    cuuint32_t b[2] = {32, 32}, estr[2] = {1, 1};
    const CUresult r = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, y, dims, strides, b, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, bf16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MAPLE_OK : MAPLE_ERR_CUDA;
}

constexpr int kRowTokens = 16;      // most tokens of linear_rows_kernel
constexpr int kRowCodes = 98304;    // and most bytes of their codes in shared memory (two CTAs on an SM)

int rows_smem(int64_t T, int K)
{
    const int NT = T <= 8 ? 1 : 2;
    return 8 * NT * row_pitch(K) + 2 * kRowWarps * NT * 512;
}
// With the norm every block reads the fp32 rows three times, which pays up to 16384
// values: into 2560 columns the two launches of the other path take 13.6 us for one
// row of 2048 and this kernel 9.4, 14.2 and 12.4 for 8 rows; into 4096 columns 21.7
// and 17.5 for 4 rows of 4096.  Above it loses: 14.4 and 21.4 for 16 rows of 2048,
// 37.1 and 39.0 for 4 of 8192.  (16 rows of 1024 are the one measured loss inside the
// rule: 10.5 and 12.2.)
bool rows_path(int64_t T, int K, bool normalise)
{
    return T <= kRowTokens && rows_smem(T, K) <= kRowCodes && (!normalise || T * K <= 16384);
}

template <int NT, bool NORM>
int launch_rows(const maple_attn_linear_args &a, const LinearOut &o, cudaStream_t st)
{
    const int smem = rows_smem(a.T, (int)a.K);
    if (smem > 49152 && cudaFuncSetAttribute(linear_rows_kernel<NT, NORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowCodes) != cudaSuccess) {
        cudaGetLastError();
        return MAPLE_ERR_CUDA;
    }
    const int64_t tiles = (a.N + 15) / 16;
    linear_rows_kernel<NT, NORM><<<(unsigned)(tiles < 2 * 148 ? tiles : 2 * 148), kRowWarps * 32, smem, st>>>(
        a.x, a.x_stride, (int)a.T, (int)a.K, a.w, o);
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}

// Tile width of the T > 128 form.  A step of 128 bytes of K writes (128 + bn) 128
// bytes into shared memory and the products read as many, at 128 bytes a clock
// together, which is more than the products' own 2 bn clocks: so the cost is the
// rounds over the 148 SMs times 128 + bn, the least over widths 64 .. 256 (4096 x
// 2560: 224 columns, 3 rounds).  Pairs of CTAs (256 x 256 tiles, each loading
// half of B) moved a third less but took 30 us against 27: 160 tiles are three
// rounds of 74 pairs.
int pick_bn(int64_t T, int64_t N)
{
    const int64_t ta = (T + 127) / 128;
    int best = 64;
    int64_t cost = -1;
    for (int bn = 64; bn <= 256; bn += 32) {
        const int64_t rounds = (ta * ((N + bn - 1) / bn) + 147) / 148, c = rounds * (128 + bn);
        if (cost < 0 || c < cost || (c == cost && bn > best)) {
            cost = c;
            best = bn;
        }
    }
    return best;
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

extern "C" int64_t maple_attn_linear_workspace(int64_t T, int64_t K, int64_t N, int32_t normalise)
{
    const int rc = check_sizes(T, K, N);
    if (rc) return rc;
    if (T == 0 || rows_path(T, (int)K, normalise != 0)) return 0;
    return round256(T * K) + round256(T * 4);   // codes and scales
}

extern "C" int maple_attn_linear(const maple_attn_linear_args *args, maple_stream_t stream)
{
    if (!args) return MAPLE_ERR_INVALID_ARG;
    const maple_attn_linear_args &a = *args;
    const int64_t need = maple_attn_linear_workspace(a.T, a.K, a.N, a.normalise);
    if (need < 0) return (int)need;
    if (a.normalise && a.K % 256) return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (a.y_dtype != MAPLE_BF16 && a.y_dtype != MAPLE_FP32) return MAPLE_ERR_INVALID_ARG;
    if (a.T == 0) return MAPLE_OK;
    if (!a.x || !a.w || !a.alpha || !a.y || (need && (!a.workspace || a.workspace_bytes < need))) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {a.x, (const void *)a.w, (const void *)a.alpha, (const void *)a.bias, (const void *)a.resid,
                          (const void *)a.y, (const void *)a.workspace})
        if (!aligned16(p)) return MAPLE_ERR_INVALID_ARG;
    if (a.x_stride % 8) return MAPLE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const int K = (int)a.K;
    const LinearOut o{a.alpha, a.bias, a.resid, a.y, a.N, a.y_dtype == MAPLE_BF16};
    if (rows_path(a.T, K, a.normalise != 0)) {
        if (a.normalise) return a.T <= 8 ? launch_rows<1, true>(a, o, st) : launch_rows<2, true>(a, o, st);
        return a.T <= 8 ? launch_rows<1, false>(a, o, st) : launch_rows<2, false>(a, o, st);
    }

    int8_t *q = (int8_t *)a.workspace;
    float *s = (float *)((char *)a.workspace + round256(a.T * a.K));
    const bool swap = a.T <= 128;
    GemmArgs p;
    memset(&p, 0, sizeof p);
    p.o = o;
    p.s = s;
    p.T = a.T;
    p.K = K;
    p.bn = swap ? (int)((a.T + 15) / 16 * 16) : pick_bn(a.T, a.N);
    p.flag = a.flags;
    p.tiles_a = ((swap ? a.N : a.T) + 127) / 128;
    p.tiles_b = ((swap ? a.T : a.N) + p.bn - 1) / p.bn;
    CUtensorMap qm, wm;
    int rc = row_map(&qm, q, a.T, K, swap ? p.bn : 128);
    if (!rc) rc = row_map(&wm, a.w, a.N, K, swap ? 128 : p.bn);
    if (rc) return rc;
    const int stage = (128 + p.bn) * kGemmBK;
    const int room = swap ? 212992 : 212992 - 40960;
    p.stages = room / stage < 8 ? room / stage : 8;
    const int smem = p.stages * stage + (swap ? 0 : 40960) + 256;
    const bool bf16 = a.y_dtype == MAPLE_BF16;
    CUtensorMap ym = qm;       // (not read without y_tma)
    p.y_tma = !swap && a.N % (bf16 ? 8 : 4) == 0;
    if (p.y_tma && (rc = out_map(&ym, a.y, a.T, a.N, bf16))) return rc;
    auto kernel = swap ? linear_gemm_kernel<true> : linear_gemm_kernel<false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024) != cudaSuccess) {
        cudaGetLastError();
        return MAPLE_ERR_CUDA;
    }
    if (a.normalise) {
        const int warps = K <= 4096 ? 4 : 1;   // (K bf16 values of shared memory a warp)
        if ((size_t)warps * K * 2 > 49152 &&
            cudaFuncSetAttribute(norm_quantise_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536) != cudaSuccess) {
            cudaGetLastError();
            return MAPLE_ERR_CUDA;
        }
        norm_quantise_rows_kernel<<<(unsigned)((a.T + warps - 1) / warps), warps * 32, (size_t)warps * K * 2, st>>>(
            (const float *)a.x, a.x_stride, a.T, K, q, s);
    } else {
        auto quantise = K <= 1024 ? quantise_rows_kernel<4> : K <= 2048 ? quantise_rows_kernel<8> : K <= 4096 ? quantise_rows_kernel<16>
                                                                                               : quantise_rows_kernel<0>;
        quantise<<<(unsigned)((a.T + 7) / 8), 256, 0, st>>>((const uint16_t *)a.x, a.x_stride, a.T, K, q, s);
    }
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    const int64_t tiles = p.tiles_a * p.tiles_b;
    lc.gridDim = dim3((unsigned)(tiles < 148 ? tiles : 148));
    lc.blockDim = dim3(kGemmThreads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaLaunchKernelEx(&lc, kernel, swap ? wm : qm, swap ? qm : wm, ym, p) != cudaSuccess) {
        cudaGetLastError();
        return MAPLE_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}
