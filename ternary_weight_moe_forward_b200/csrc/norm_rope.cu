// Per-head RMS norm of queries and keys, rotation by position and the append
// to the 4-bit cache in one pass; reading cached rows back.  C ABI:
// include/maple_attn.h.
#include <stdint.h>

#include "../../include/maple_attn.h"
#include "kv_cache.cuh"

using namespace maple;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// A head is held by D/8 lanes, 8 channels (16 bytes) each, so that the norm is a
// sum over these lanes, the rotation partner of a lane's channels sits in one
// other lane (pairs half a rotation apart) or in the lane itself (neighbours),
// and a group of 32 cached channels is 4 lanes, each writing one word of codes.
// A token is split over `parts` warps (one for long prompts, as many as it has
// head groups for a single token); each computes the token's angles once, under
// its first loads, and keeps them in its own shared memory, so that no warp
// waits for another.  kAhead loads of 16 bytes per lane are in flight.
//
// Angle: position * inv_freq in units of whole turns, in 64 bits (a product of
// 10^6 radians has lost all of its fraction's accuracy in 32), reduced to
// [-1/2, 1/2] turns before the 32-bit sine and cosine.
//
// Bound: HBM traffic for long prompts (each head is read and written once),
// latency for one token.  One CTA per token with a barrier behind the angles
// took 66 us for 16384 tokens of 36 heads of 64.
constexpr int kRopeWarps = 4, kAhead = 2;

template <typename T, int D, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kRopeWarps * 32, 8) qk_norm_rope_kernel(const maple_attn_rope_args a, const int parts)
{
    using P = KvPage<D>;
    constexpr int LPH = D / 8, HPW = 32 / LPH;      // lanes of a head, heads of a warp's step
    __shared__ __align__(16) float s_angle[kRopeWarps][2][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPH;
    float *cs = s_angle[warp][0], *sn = s_angle[warp][1];
    const int H = a.heads, Hkv = a.kv_heads, rd = a.rotary_dim, half = rd >> 1;
    const int U = H + Hkv + (CACHE ? Hkv : 0), steps = (U + HPW - 1) / HPW;
    const int n = a.page_size;
    const int64_t jobs = a.T * parts, nw = (int64_t)gridDim.x * kRopeWarps;

  for (int64_t job = blockIdx.x * (int64_t)kRopeWarps + warp; job < jobs; job += nw) {
    const int64_t t = job / parts;
    const int part = (int)(job - t * parts);
    // head u of q, k and v is at base + u D
    const T *bq = (const T *)a.q + t * a.q_stride + 8 * l;
    const T *bk = (const T *)a.k + t * a.k_stride + 8 * l - (int64_t)H * D;
    const T *bv = CACHE ? (const T *)a.v + t * a.v_stride + 8 * l - (int64_t)(H + Hkv) * D : bk;
    auto source = [&](int u) { return reinterpret_cast<const uint4 *>((u < H ? bq : u < H + Hkv ? bk : bv) + u * D); };
    uint4 ahead[kAhead];
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int st = s0 + i * parts, u = st * HPW + lane / LPH;
            ahead[i] = st < steps && u < U ? __ldg(source(u)) : make_uint4(0, 0, 0, 0);
        }
    };
    load(part);
    int64_t slot = -1;
    if (CACHE) {
        slot = __ldg(a.slots + t);
        if (slot >= a.num_pages * n) {
            if (lane == 0) set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
            slot = -1;
        }
    }
    const double pos = rd ? (double)__ldg(a.positions + t) : 0.0;
    __syncwarp();      // (the last job's angles are read)
    for (int i = lane; i < half; i += 32) {
        double turns = pos * (__ldg(a.inv_freq + i) * 0.15915494309189533577);
        turns -= rint(turns);
        sincospif(2.0f * (float)turns, &sn[i], &cs[i]);
    }
    __syncwarp();

    const int64_t page = slot >= 0 ? slot / n : 0;
    const int row = slot >= 0 ? (int)(slot - page * n) : 0;
    for (int s0 = part; s0 < steps; s0 += kAhead * parts) {
      uint4 now[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; i++) now[i] = ahead[i];
      load(s0 + kAhead * parts);
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int st = s0 + i * parts, u = st * HPW + lane / LPH;
        if (st >= steps) break;
        const bool on = u < U;
        float x[8];
        unpack8<T>(now[i], x);
        // ---- norm (the heads of q and k)
        float ss = 0.0f;
#pragma unroll
        for (int m = 0; m < 8; m++) ss = fmaf(x[m], x[m], ss);
#pragma unroll
        for (int o = LPH / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
        const bool qk = u < H + Hkv;
        if (qk) {
            const float inv = rsqrtf(ss * (1.0f / D) + a.eps);   // (2 ulp)
            const float *wt = u < H ? a.q_weight : a.k_weight;
            if (wt) {
                const float4 w0 = __ldg(reinterpret_cast<const float4 *>(wt) + 2 * l);
                const float4 w1 = __ldg(reinterpret_cast<const float4 *>(wt) + 2 * l + 1);
                const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int m = 0; m < 8; m++) x[m] = x[m] * inv * w[m];
            } else {
#pragma unroll
                for (int m = 0; m < 8; m++) x[m] *= inv;
            }
        }
        // ---- rotation
        const int c0 = 8 * l;
        if (INTER) {
            if (qk && c0 < rd) {
                const float4 c4 = reinterpret_cast<const float4 *>(cs)[l], s4 = reinterpret_cast<const float4 *>(sn)[l];
                const float cv[4] = {c4.x, c4.y, c4.z, c4.w}, sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int m = 0; m < 8; m += 2) {
                    const float c = cv[m / 2], s = sv[m / 2], x0 = x[m], x1 = x[m + 1];
                    x[m] = fmaf(x0, c, -(x1 * s));
                    x[m + 1] = fmaf(x1, c, x0 * s);
                }
            }
        } else if (rd) {
            const bool first = c0 < half;
            const int src = c0 < rd ? (first ? lane + half / 8 : lane - half / 8) : lane;
            float y[8];
#pragma unroll
            for (int m = 0; m < 8; m++) y[m] = __shfl_sync(FULL, x[m], src);
            if (qk && c0 < rd) {
                const int i4 = (first ? c0 : c0 - half) / 4;
                const float sign = first ? -1.0f : 1.0f;
#pragma unroll
                for (int z = 0; z < 2; z++) {
                    const float4 c4 = reinterpret_cast<const float4 *>(cs)[i4 + z], s4 = reinterpret_cast<const float4 *>(sn)[i4 + z];
                    x[4 * z] = fmaf(x[4 * z], c4.x, y[4 * z] * (sign * s4.x));
                    x[4 * z + 1] = fmaf(x[4 * z + 1], c4.y, y[4 * z + 1] * (sign * s4.y));
                    x[4 * z + 2] = fmaf(x[4 * z + 2], c4.z, y[4 * z + 2] * (sign * s4.z));
                    x[4 * z + 3] = fmaf(x[4 * z + 3], c4.w, y[4 * z + 3] * (sign * s4.w));
                }
            }
        }
        const uint4 out = pack8<T>(x);
        if (on && u < H) reinterpret_cast<uint4 *>((T *)a.q_out + (t * H + u) * D)[l] = out;
        else if (on && qk && a.k_out) reinterpret_cast<uint4 *>((T *)a.k_out + (t * Hkv + (u - H)) * D)[l] = out;
        if (!CACHE || !__any_sync(FULL, on && u >= H && slot >= 0)) continue;
        // ---- 4-bit codes of the keys (as rounded) and values
        unpack8<T>(out, x);   // (a value is its own rounding)
        float lo = kKvClamp, hi = -kKvClamp;
        bool nan = false;
#pragma unroll
        for (int m = 0; m < 8; m++) {
            nan = nan || x[m] != x[m];
            x[m] = fminf(fmaxf(x[m], -kKvClamp), kKvClamp);
            lo = fminf(lo, x[m]);
            hi = fmaxf(hi, x[m]);
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(FULL, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(FULL, hi, o));
            nan = __shfl_xor_sync(FULL, (int)nan, o) || nan;
        }
        const __half mh = nan ? __ushort_as_half(0x7fff) : __float2half_rn(lo);
        const float mf = __half2float(mh);
        const __half sh = nan ? __ushort_as_half(0x7fff) : __float2half_rn(__fdiv_rn(hi - mf, 15.0f));
        const float sf = __half2float(sh);
        uint32_t word = 0;
        if (sf > 0.0f) {
#pragma unroll
            for (int m = 0; m < 8; m++) {
                const int c = min(15, max(0, __float2int_rn(__fdiv_rn(x[m] - mf, sf))));
                word |= (uint32_t)c << (4 * m);
            }
        }
        if (on && u >= H && slot >= 0) {
            const bool key = u < H + Hkv;
            const int h = key ? u - H : u - H - Hkv, g = l >> 2;
            uint8_t *base = a.pages + (page * Hkv + h) * P::bytes(n);
            *reinterpret_cast<uint32_t *>(base + (key ? P::k_word(row, l) : P::v_word(n, row, l))) = word;
            if ((l & 3) == 0) {
                if (key) {
                    *reinterpret_cast<__half2 *>(base + P::k_pair(n, row, g)) = __halves2half2(sh, mh);
                } else {
                    *reinterpret_cast<__half *>(base + P::v_scale(n, row, g)) = sh;
                    *reinterpret_cast<__half *>(base + P::v_min(n, row, g)) = mh;
                }
            }
        }
      }
    }
  }
}

// One thread per (slot, head, 8 channels): one word of codes and the group's
// pair of K, the same of V, one 16-byte store each.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const maple_attn_read_args a)
{
    using P = KvPage<D>;
    constexpr int W = D / 8;
    const int64_t total = a.n * a.kv_heads * W;
    const int n = a.page_size;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int w = (int)(i % W);
        const int64_t th = i / W, t = th / a.kv_heads;
        const int h = (int)(th - t * a.kv_heads);
        const int64_t slot = __ldg(a.slots + t);
        uint4 ko = make_uint4(0, 0, 0, 0), vo = ko;
        if (slot >= a.num_pages * n) {
            set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
        } else if (slot >= 0) {
            const int64_t page = slot / n;
            const int p = (int)(slot - page * n), g = w >> 2;
            const uint8_t *base = a.pages + (page * a.kv_heads + h) * P::bytes(n);
            const uint32_t kw = *reinterpret_cast<const uint32_t *>(base + P::k_word(p, w));
            const uint32_t vw = *reinterpret_cast<const uint32_t *>(base + P::v_word(n, p, w));
            const float2 kp = __half22float2(*reinterpret_cast<const __half2 *>(base + P::k_pair(n, p, g)));
            const float vs = __half2float(*reinterpret_cast<const __half *>(base + P::v_scale(n, p, g)));
            const float vm = __half2float(*reinterpret_cast<const __half *>(base + P::v_min(n, p, g)));
            float k[8], v[8];
#pragma unroll
            for (int m = 0; m < 8; m++) {
                k[m] = fmaf(kp.x, (float)((kw >> (4 * m)) & 15u), kp.y);   // (the product is exact)
                v[m] = fmaf(vs, (float)((vw >> (4 * m)) & 15u), vm);
            }
            ko = pack8<T>(k);
            vo = pack8<T>(v);
        }
        reinterpret_cast<uint4 *>(a.k)[i] = ko;
        reinterpret_cast<uint4 *>(a.v)[i] = vo;
    }
}

template <int V>
struct Int {
    static constexpr int value = V;
};

bool heads_ok(int H, int Hkv) { return H >= 1 && Hkv >= 1 && H <= 1024 && H % Hkv == 0; }

}  // namespace

extern "C" int64_t maple_attn_page_bytes(int32_t head_dim, int32_t page_size)
{
    if ((head_dim != 64 && head_dim != 128) || (page_size != 16 && page_size != 32 && page_size != 64))
        return MAPLE_ERR_UNSUPPORTED_SHAPE;
    return (int64_t)page_size * head_dim * 5 / 4;
}

extern "C" int maple_attn_qk_norm_rope(const maple_attn_rope_args *args, maple_stream_t stream)
{
    if (!args) return MAPLE_ERR_INVALID_ARG;
    const maple_attn_rope_args &a = *args;
    const int D = a.head_dim;
    if ((D != 64 && D != 128) || !heads_ok(a.heads, a.kv_heads) || a.rotary_dim < 0 || a.rotary_dim > D ||
        a.rotary_dim % 16)
        return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (a.pages && maple_attn_page_bytes(D, a.page_size) < 0) return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (a.dtype != MAPLE_BF16 && a.dtype != MAPLE_FP16) return MAPLE_ERR_INVALID_ARG;
    if (a.T < 0 || a.T > 0x7fffffffll || !(a.eps >= 0.0f)) return MAPLE_ERR_INVALID_ARG;
    if (a.T == 0) return MAPLE_OK;
    if (!a.q || !a.k || !a.q_out || (!a.k_out && !a.pages)) return MAPLE_ERR_INVALID_ARG;
    if (a.rotary_dim && (!a.positions || !a.inv_freq)) return MAPLE_ERR_INVALID_ARG;
    if (a.pages && (!a.v || !a.slots || a.num_pages < 1 || a.num_pages > (1ll << 40))) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {a.q, a.k, a.pages ? a.v : nullptr, (const void *)a.q_out, (const void *)a.k_out,
                          (const void *)a.q_weight, (const void *)a.k_weight, (const void *)a.pages})
        if (!aligned16(p)) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {(const void *)a.positions, (const void *)a.inv_freq, (const void *)a.slots})
        if ((uintptr_t)p & 7u) return MAPLE_ERR_INVALID_ARG;
    if (a.q_stride % 8 || a.k_stride % 8 || (a.pages && a.v_stride % 8)) return MAPLE_ERR_INVALID_ARG;
    // warps of a token: enough to give every SM some for few tokens, one for many
    const int U = a.heads + a.kv_heads * (a.pages ? 2 : 1), steps = (U * (D / 8) + 31) / 32;
    const int64_t want = 148 * 16 / a.T;
    const int parts = (int)(want < 1 ? 1 : want > steps ? steps : want);
    const int64_t blocks = (a.T * parts + kRopeWarps - 1) / kRopeWarps;
    const unsigned grid = (unsigned)(blocks < 148 * 16 ? blocks : 148 * 16);
    const int threads = kRopeWarps * 32;
    cudaStream_t st = (cudaStream_t)stream;
    auto launch = [&](auto elem, auto dim) {
        using T = decltype(elem);
        constexpr int DIM = decltype(dim)::value;
        auto kernel = a.interleaved ? (a.pages ? qk_norm_rope_kernel<T, DIM, true, true> : qk_norm_rope_kernel<T, DIM, true, false>)
                                    : (a.pages ? qk_norm_rope_kernel<T, DIM, false, true> : qk_norm_rope_kernel<T, DIM, false, false>);
        kernel<<<grid, threads, 0, st>>>(a, parts);
    };
    if (a.dtype == MAPLE_BF16) {
        if (D == 128) launch(__nv_bfloat16(), Int<128>());
        else launch(__nv_bfloat16(), Int<64>());
    } else {
        if (D == 128) launch(__half(), Int<128>());
        else launch(__half(), Int<64>());
    }
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}

extern "C" int maple_attn_kv_read(const maple_attn_read_args *args, maple_stream_t stream)
{
    if (!args) return MAPLE_ERR_INVALID_ARG;
    const maple_attn_read_args &a = *args;
    if (maple_attn_page_bytes(a.head_dim, a.page_size) < 0 || a.kv_heads < 1 || a.kv_heads > 1024)
        return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (a.dtype != MAPLE_BF16 && a.dtype != MAPLE_FP16) return MAPLE_ERR_INVALID_ARG;
    if (a.n < 0 || a.n > 0x7fffffffll) return MAPLE_ERR_INVALID_ARG;
    if (a.n == 0) return MAPLE_OK;
    if (!a.pages || !a.slots || !a.k || !a.v || a.num_pages < 1 || a.num_pages > (1ll << 40) || !aligned16(a.pages) ||
        !aligned16(a.k) || !aligned16(a.v) || ((uintptr_t)a.slots & 7u))
        return MAPLE_ERR_INVALID_ARG;
    const int64_t total = a.n * a.kv_heads * (a.head_dim / 8);
    const int64_t blocks = (total + 255) / 256;
    const int grid = (int)(blocks < 148 * 32 ? blocks : 148 * 32);
    cudaStream_t st = (cudaStream_t)stream;
    if (a.dtype == MAPLE_BF16) {
        if (a.head_dim == 128) kv_read_kernel<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(a);
        else kv_read_kernel<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(a);
    } else {
        if (a.head_dim == 128) kv_read_kernel<__half, 128><<<grid, 256, 0, st>>>(a);
        else kv_read_kernel<__half, 64><<<grid, 256, 0, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}
