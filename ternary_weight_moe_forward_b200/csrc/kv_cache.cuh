// The paged cache of 4-bit keys and values: byte layout of a page of one head
// and the helpers shared by the kernels that write and read it.
//
// A token and head holds d codes of 4 bits for K and for V and one (scale,
// minimum) pair of fp16 per 32 channels: 1.25 d bytes against the 4 d of bf16.
// value = minimum + scale * code.  Groups of 32 keep the pairs at a fifth of
// the bytes; one pair per token (not per channel) lets a token be appended
// without touching its neighbours.
//
// The order of the bytes is the one in which the lanes of m16n8k16 matrix
// instructions want them (cached_attention reads whole pages with bulk copies
// and takes its fragments from shared memory without a shuffle or a bank
// conflict).  "word w" = the 8 codes of channels 8w .. 8w+7, channel 8w+i in
// bits 4i .. 4i+3.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace maple {

constexpr float kKvClamp = 60000.0f;   // minimum + 15 * scale stays a finite fp16

template <int D>
struct KvPage {
    static constexpr int kGroups = D / 32;
    static constexpr int kRowBytes = D + D / 4;              // K and V codes, K and V pairs of a token and head
    static __host__ __device__ constexpr int bytes(int n) { return n * kRowBytes; }
    // byte offsets in a page of n rows
    static __host__ __device__ constexpr int k_word(int p, int w) { return p * (D / 2) + ((w & 3) * kGroups + (w >> 2)) * 4; }
    static __host__ __device__ constexpr int v_word(int n, int p, int w)
    {
        const int r = p & 15, u = (r & 7) >> 1, z = (r & 1) + 2 * (r >> 3);
        const int blk = n * (D / 2) + (p >> 4) * (8 * D);
        return D == 128 ? blk + (z >> 1) * 512 + ((w >> 1) * 4 + u) * 16 + (z & 1) * 8 + (w & 1) * 4
                        : blk + (w * 4 + u) * 16 + z * 4;
    }
    static __host__ __device__ constexpr int k_pair(int n, int p, int g) { return n * D + (p * kGroups + g) * 4; }
    static __host__ __device__ constexpr int v_scale(int n, int p, int g) { return n * D + n * kGroups * 4 + (g * n + p) * 2; }
    static __host__ __device__ constexpr int v_min(int n, int p, int g) { return v_scale(n, p, g) + n * kGroups * 2; }
};

// element types: conversions to and from fp32 (one rounding), two at a time
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = Elem<T>::unpack(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]), Elem<T>::pack(x[4], x[5]),
                      Elem<T>::pack(x[6], x[7]));
}

}  // namespace maple
