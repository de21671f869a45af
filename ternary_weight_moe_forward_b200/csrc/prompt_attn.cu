// Causal attention over packed prompts on the 5th-generation tensor cores.
// C ABI: include/maple_attn.h.
//
// Mathematics.  S = Q K^T and O += P V on tcgen05 (kind::f16, M = 128, fp32
// accumulators in tensor memory), P = 2^(scale2 S - m) with a running reference
// m per row and the row sum l beside it, out = O / l.  The reference follows
// the row maximum only when a score passes it by 2^8: until then P stays below
// 256, the sums stay exact in the same way, and O need not be rescaled.  P is
// rounded to the inputs' type (the tensor cores' operand); l sums it before the
// rounding.
//
// Rows.  A tile is 128 rows = floor(128/G) query tokens x the G query heads of
// one key/value head, so that grouped heads share every K and V tile (one 3-D
// TMA box brings them, whatever G), and a short prompt fills a tile with heads.
//
// One CTA works on two tiles (A and B, consecutive tokens) of a sequence and a
// key/value head, over tiles of 128 keys:
//   warp 8    TMA: Q once, then K_0, V_0, K_1, V_1, ... into a ring
//   warp 9    MMA: S_A = Q_A K_0, S_B = Q_B K_0, then per key tile j
//             O_A += P_A V_j, S_A = Q_A K_j+1, O_B += P_B V_j, S_B = Q_B K_j+1
//   warps 0-3 softmax of A, warps 4-7 of B: one thread per row, S from tensor
//             memory, P back over the same columns; rescaling and the epilogue
// While one tile's rows are in the exponentials, the tensor cores work on the
// other's products.  Tensor memory: S_A, S_B (P over their first half), O_A,
// O_B = 512 columns at d = 128.  In-order execution of the MMAs makes "S_j full"
// imply that O has taken V_j-1.
//
// Masked keys.  P is 0 there, but 0 times an infinity or NaN in V would reach
// the sums; so tiles that hold masked keys have what is not finite in V set to
// 0 in shared memory first, and if anything was found the rows that do see
// those values add them again at the end.
//
// Work is ordered from the last tokens (the longest rows) to the first, so that
// the short items fill the end of the run.
#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include "../../include/maple_attn.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

using namespace maple;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// three warpgroups: two of softmax rows, one of which two warps work; the
// launch's 384 x 168 registers are shared out as 2 x 128 x 216 + 128 x 72
constexpr int kThreads = 384;
constexpr int kKeys = 128;   // keys of a tile

template <int D>
struct PromptSmem {
    static constexpr int kHalves = D / 64;                 // 64-column (128-byte) sub-tiles
    static constexpr int kTileBytes = kHalves * 128 * 128; // a Q, K or V tile
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kKv = 2 * kTileBytes;             // after Q_A and Q_B
    static constexpr int kBars = kKv + kStages * kTileBytes;
    static constexpr int kTotal = kBars + 512;
};

struct PromptK {
    maple_attn_prompt_args a;
    int G, nt;                 // query heads of a key/value head, tokens of a tile
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tcgen05 kind::f16: bf16 or fp16 operands, fp32 accumulator, M = 128; B either
// K-major (keys as rows of K) or MN-major (V: its rows are the K dimension)
__device__ __forceinline__ uint32_t idesc_f16(bool bf16, int n, bool b_mn)
{
    const uint32_t f = bf16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// MN-major operand, 128-byte swizzle: rows (K index) of 64 values, 8-row atoms
// 1024 bytes apart, the next 64 values of a row 16 KB further
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(16384 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// the bits of the two 16-bit halves of w that hold an infinity or NaN
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t E = sizeof(T) && __is_same(T, __nv_bfloat16) ? 0x7f80u : 0x7c00u;
    return ((w & E) == E ? 0xffffu : 0u) | ((w & (E << 16)) == (E << 16) ? 0xffff0000u : 0u);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptK p)
{
    using L = PromptSmem<D>;
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int s_item[8];
    __shared__ int s_warp[kThreads / 32];
    const maple_attn_prompt_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_addr(smem) & 1023u) {   // the swizzled tiles need 1024-byte alignment
        if (threadIdx.x == 0) set_flag(a.flags, MAPLE_DEVFLAG_TIMEOUT);
        return;
    }
    uint64_t *bars = (uint64_t *)(smem + L::kBars);
    const uint32_t b_full = smem_addr(bars), b_empty = b_full + 8 * S, b_q = b_empty + 8 * S;
    const uint32_t b_s = b_q + 8, b_p = b_s + 16, b_o = b_p + 16, b_drain = b_o + 16;
    uint32_t *tmem_holder = (uint32_t *)(bars + 2 * S + 8);
    volatile uint32_t *abort = tmem_holder + 1;
    uint32_t *odd_values = tmem_holder + 2;   // something in V was not finite

    // ---- this CTA's item: sequence, pair of tiles; items lie sequence by
    // sequence, taken from the end
    const int span = 2 * p.nt;
    const int item_kv = blockIdx.x % a.kv_heads, kvh = item_kv;
    const int x = blockIdx.x / a.kv_heads;
    auto bounds = [&](int b, int64_t &q0, int64_t &q1, bool &bad) {
        const int64_t u = __ldg(a.cu_q + b), v = __ldg(a.cu_q + b + 1);
        q0 = min(max(u, (int64_t)0), a.Tq);
        q1 = min(max(v, q0), a.Tq);
        bad = q0 != u || q1 != v || q1 - q0 > a.max_q;
        q1 = min(q1, q0 + a.max_q);
    };
    if (threadIdx.x == 0) {
        s_item[0] = -1;
        for (int s = 0; s < S; s++) {
            mbar_init(b_full + 8 * s, 1);
            mbar_init(b_empty + 8 * s, 1);
        }
        mbar_init(b_q, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_p + 8 * i, 4);
            mbar_init(b_o + 8 * i, 1);
        }
        mbar_init(b_drain, 1);
        *abort = 0u;
        *odd_values = 0u;
        fence_barrier_init();
    }
    // count the pairs from the last sequence on; the thread whose stretch of sequences holds item x finds it
    {
        const int per = (a.B + kThreads - 1) / kThreads;
        const int hi = a.B - min((int)threadIdx.x * per, a.B), lo = max(hi - per, 0);
        int mine = 0;
        for (int b = hi - 1; b >= lo; b--) {
            int64_t q0, q1;
            bool bad;
            bounds(b, q0, q1, bad);
            mine += (int)((q1 - q0 + span - 1) / span);
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        int at = inc - mine;
        for (int w = 0; w < warp; w++) at += s_warp[w];
        if (x >= at && x < at + mine) {
            for (int b = hi - 1; b >= lo; b--) {
                int64_t q0, q1;
                bool bad;
                bounds(b, q0, q1, bad);
                const int n = (int)((q1 - q0 + span - 1) / span);
                if (x >= at && x < at + n) {
                    const int64_t ku = __ldg(a.cu_k + b), kv = __ldg(a.cu_k + b + 1);
                    const int64_t k0 = min(max(ku, (int64_t)0), a.Tk), k1 = min(max(kv, k0), a.Tk);
                    s_item[0] = n - 1 - (x - at);   // the last tokens first
                    s_item[1] = (int)q0;
                    s_item[2] = (int)(q1 - q0);
                    s_item[3] = (int)k0;
                    s_item[4] = (int)(k1 - k0);
                    // (the cut of max_q does not move the queries' positions)
                    s_item[5] = (int)((k1 - k0) - (min(max((int64_t)__ldg(a.cu_q + b + 1), q0), a.Tq) - q0));
                }
                at += n;
            }
        }
        if (blockIdx.x == 0) {   // report offsets that were cut
            for (int b = hi - 1; b >= lo; b--) {
                int64_t q0, q1;
                bool bad;
                bounds(b, q0, q1, bad);
                const int64_t ku = __ldg(a.cu_k + b), kv = __ldg(a.cu_k + b + 1);
                if (bad || ku < 0 || kv < ku || kv > a.Tk) set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
            }
        }
    }
    __syncthreads();
    const int pair = s_item[0];
    if (pair < 0) return;       // beyond the last item
    const int q0 = s_item[1], lq = s_item[2], k0 = s_item[3], off = s_item[5];
    const int tA = pair * span, tB = tA + p.nt;
    const bool hasB = tB < lq;
    const int last = min(tA + span, lq) - 1;               // last query token of the pair
    const int kbeg = a.window ? max(tA + off - a.window + 1, 0) : 0, kend = last + off + 1;
    const int n = kend > kbeg ? (kend - kbeg + kKeys - 1) / kKeys : 0;   // tiles of keys
    // whether some row of the pair does not see all keys of tile j
    auto masked = [&](int j) {
        const int s = kbeg + j * kKeys;
        return s + kKeys - 1 > tA + off || (a.window && s < last + off - a.window + 1);
    };

    if (warp == 9) tmem_alloc(smem_addr(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    constexpr uint32_t kO = 256;   // first column of O_A
    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp == 8) {
        // ---------------- loads
        if (lane == 0 && n > 0) {
            mbar_expect_tx(b_q, (hasB ? 2 : 1) * L::kHalves * p.G * p.nt * 128);
            for (int i = 0; i < (hasB ? 2 : 1); i++)
                for (int h = 0; h < L::kHalves; h++)
                    tma_load_3d(smem_addr(smem + i * L::kTileBytes + h * 16384), &q_map, 64 * h, kvh * p.G, q0 + (i ? tB : tA), b_q);
            int it = 0;
            bool ok = true;
            for (; it < 2 * n; it++) {
                const int s = it % S;
                if (!mbar_wait(b_empty + 8 * s, ((it / S) & 1) ^ 1, abort, a.flags, kDefaultWaitNs)) {
                    ok = false;
                    break;
                }
                mbar_expect_tx(b_full + 8 * s, L::kTileBytes);
                for (int h = 0; h < L::kHalves; h++)
                    tma_load_3d(smem_addr(smem + L::kKv + s * L::kTileBytes + h * 16384), (it & 1) ? &v_map : &k_map, 64 * h, kvh,
                                k0 + kbeg + (it >> 1) * kKeys, b_full + 8 * s);
            }
            if (!ok) {   // drain the copies in flight
                for (int j = it > S ? it - S : 0; j < it; j++) {
                    const uint64_t t0 = global_ns();
                    while (!mbar_test(b_full + 8 * (j % S), (j / S) & 1) && global_ns() - t0 < kDefaultWaitNs) {
                    }
                }
                const uint64_t t0 = global_ns();
                while (!mbar_test(b_q, 0) && global_ns() - t0 < kDefaultWaitNs) {
                }
            }
        }
      } else if (warp == 9) {
        // ---------------- products
        if (lane == 0 && n > 0) {
            const bool bf = __is_same(T, __nv_bfloat16);
            const uint32_t id_s = idesc_f16(bf, kKeys, false), id_o = idesc_f16(bf, D, true);
            bool ok = mbar_wait(b_q, 0, abort, a.flags, kDefaultWaitNs);
            auto wait_tile = [&](int it) { return mbar_wait(b_full + 8 * (it % S), (it / S) & 1, abort, a.flags, kDefaultWaitNs); };
            auto scores = [&](int i, int j) {   // S_i = Q_i K_j^T
                const uint32_t kb = smem_addr(smem + L::kKv + ((2 * j) % S) * L::kTileBytes);
                const uint64_t da = desc_sw128(smem_addr(smem + i * L::kTileBytes)), db = desc_sw128(kb);
#pragma unroll
                for (int k = 0; k < D / 16; k++)
                    mma_ss(tmem + 128 * i, da + (k / 4) * 1024 + 2 * (k % 4), db + (k / 4) * 1024 + 2 * (k % 4), id_s, k != 0);
                mma_commit(b_s + 8 * i);
            };
            auto values = [&](int i, int j) {   // O_i += P_i V_j
                const uint64_t db = desc_mn_sw128(smem_addr(smem + L::kKv + ((2 * j + 1) % S) * L::kTileBytes));
#pragma unroll
                for (int k = 0; k < kKeys / 16; k++)
                    mma_ts(tmem + kO + D * i, tmem + 128 * i + 8 * k, db + 128 * k, id_o, (j | k) != 0);
            };
            const int ni = hasB ? 2 : 1;
            if (ok && (ok = wait_tile(0))) {
                tc_fence_after();
                for (int i = 0; i < ni; i++) scores(i, 0);
                mma_commit(b_empty);
            }
            for (int j = 0; ok && j < n; j++) {
                ok = wait_tile(2 * j + 1) && (j + 1 == n || wait_tile(2 * j + 2));
                for (int i = 0; ok && i < ni; i++) {
                    if (!(ok = mbar_wait(b_p + 8 * i, j & 1, abort, a.flags, kDefaultWaitNs))) break;
                    tc_fence_after();
                    values(i, j);
                    if (j + 1 < n) scores(i, j + 1);
                    else mma_commit(b_o + 8 * i);
                }
                mma_commit(b_empty + 8 * ((2 * j + 1) % S));
                if (j + 1 < n) mma_commit(b_empty + 8 * ((2 * j + 2) % S));
            }
            mma_commit(b_drain);   // every issued MMA has finished before tensor memory is released
            const uint64_t t0 = global_ns();
            while (!mbar_test(b_drain, 0) && global_ns() - t0 < kDefaultWaitNs) {
            }
        }
      }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      if (warp < 4 || hasB) {
        // ---------------- softmax and epilogue: one thread per row
        const int i = warp >> 2, r = threadIdx.x & 127;
        const int tok = (i ? tB : tA) + r / p.G, h = r % p.G;
        const bool valid = r < p.G * p.nt && tok < lq;
        const int pos = tok + off;                    // key position of the row's query
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + 128 * i + lanes, to = tmem + kO + D * i + lanes;
        const bool neg = a.scale < 0.0f;
        const float scale2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);   // (0 as 10^-30: -inf stays -inf)
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < n; j++) {
            const bool edge = masked(j);
            if (edge && i == 0) {
                // V_j: what is not finite becomes 0 before the products read it
                if (!mbar_wait(b_full + 8 * ((2 * j + 1) % S), ((2 * j + 1) / S) & 1, abort, a.flags, kDefaultWaitNs)) ok = false;
                if (ok) {
                    uint4 *tile = (uint4 *)(smem + L::kKv + ((2 * j + 1) % S) * L::kTileBytes);
                    bool any = false;
#pragma unroll 4
                    for (int c = threadIdx.x; c < L::kTileBytes / 16; c += 128) {
                        const uint4 v = tile[c];
                        const uint32_t e0 = not_finite<T>(v.x), e1 = not_finite<T>(v.y), e2 = not_finite<T>(v.z), e3 = not_finite<T>(v.w);
                        if (e0 | e1 | e2 | e3) {
                            tile[c] = make_uint4(v.x & ~e0, v.y & ~e1, v.z & ~e2, v.w & ~e3);
                            any = true;
                        }
                    }
                    if (any) atomicOr(odd_values, 1u);
                    fence_async_smem();
                }
            }
            ok = ok && mbar_wait(b_s + 8 * i, j & 1, abort, a.flags, kDefaultWaitNs);
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            tc_fence_after();
            float s[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) tmem_ld32(ts + c, *reinterpret_cast<int(*)[32]>(&s[c]));
            tmem_wait_ld();
            if (neg) {
#pragma unroll
                for (int c = 0; c < kKeys; c++) s[c] = -s[c];
            }
            if (edge) {
                const int base = kbeg + j * kKeys, hi = pos - base, lo = a.window ? pos - a.window + 1 - base : -1;
#pragma unroll
                for (int c = 0; c < kKeys; c++)
                    if (c > hi || c < lo) s[c] = -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < kKeys; c++) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale2;
            const bool up = mt > m + 8.0f;
            if (__any_sync(FULL, up)) {
                const float f = !up ? 1.0f : (m == -INFINITY ? 0.0f : ex2(m - mt));
                if (up) m = mt;
                l *= f;
                if (j > 0) {
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + c, *reinterpret_cast<int(*)[32]>(o));
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(to + c, o);
                    }
                }
            }
            const float minus = m == -INFINITY ? 0.0f : -m;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < kKeys; c += 64) {
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    const float p0 = ex2(fmaf(s[c + e], scale2, minus)), p1 = ex2(fmaf(s[c + e + 1], scale2, minus));
                    sum[e & 2] += p0;
                    sum[(e & 2) + 1] += p1;
                    pk[e / 2] = Elem<T>::pack(p0, p1);
                }
                tmem_st32(ts + c / 2, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_p + 8 * i);
        }
        if (n > 0) ok = ok && mbar_wait(b_o + 8 * i, 0, abort, a.flags, kDefaultWaitNs);
        ok = __all_sync(FULL, ok);
        tc_fence_after();
        const bool fix = ok && n > 0 && *(volatile uint32_t *)odd_values != 0;
        const float inv = l > 0.0f || l != l ? __fdiv_rn(1.0f, l) : 0.0f;
        const int64_t row = (int64_t)(q0 + tok) * a.heads + kvh * p.G + h;
        if (ok) {
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(to + c, *reinterpret_cast<int(*)[32]>(o));
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e++) o[e] = 0.0f;
                }
                if (fix && valid) {
                    // the values that were set to 0 and that this row does see
                    const int from = max(a.window ? pos - a.window + 1 : 0, 0);
                    for (int j = 0; j < n; j++) {
                        if (!masked(j)) continue;
                        const int s0 = max(kbeg + j * kKeys, from), s1 = min(kbeg + (j + 1) * kKeys, pos + 1);
                        for (int key = s0; key < s1; key++) {
                            const T *v = (const T *)a.v + (int64_t)(k0 + key) * a.v_stride + (int64_t)kvh * D + c;
#pragma unroll
                            for (int e = 0; e < 32; e++) {
                                const float f = (float)v[e];
                                if (!isfinite(f)) o[e] += f;
                            }
                        }
                    }
                }
                if (valid) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float y[8];
#pragma unroll
                        for (int z = 0; z < 8; z++) y[z] = l == 0.0f ? 0.0f : o[e + z] * inv;
                        *reinterpret_cast<uint4 *>((T *)a.out + row * D + c + e) = pack8<T>(y);
                    }
                }
            }
            if (valid && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

typedef CUresult (*encode_fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [T][heads][d] with boxes of 64 channels x `bh` heads x `bt` tokens, 128-byte swizzle
int head_map(CUtensorMap *map, const void *base, int dtype, int64_t T, int heads, int d, int64_t stride, int bh, int bt)
{
    static encode_fn encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (encode_fn)fn;
    }();
    if (!encode) return MAPLE_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)bt}, estr[3] = {1, 1, 1};
    const CUresult r = encode(map, dtype == MAPLE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MAPLE_OK : MAPLE_ERR_CUDA;
}

template <typename T, int D>
int launch(const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const PromptK &k, int64_t items, cudaStream_t st)
{
    if (cudaFuncSetAttribute(prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptSmem<D>::kTotal) != cudaSuccess) {
        cudaGetLastError();
        return MAPLE_ERR_CUDA;
    }
    prompt_kernel<T, D><<<(unsigned)items, kThreads, PromptSmem<D>::kTotal, st>>>(qm, km, vm, k);
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
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
    if (a.B < 0 || a.B > 65535 || a.max_q < 0 || a.window < 0 || a.Tq < 0 || a.Tk < 0 || a.Tq > (1ll << 30) ||
        a.Tk > (1ll << 30) || !isfinite(a.scale))
        return MAPLE_ERR_INVALID_ARG;
    if (a.B == 0 || a.Tq == 0 || a.max_q == 0) return MAPLE_OK;
    if (!a.q || !a.out || !a.cu_q || !a.cu_k || (a.Tk && (!a.k || !a.v))) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {a.q, a.k, a.v, (const void *)a.out})
        if (!aligned16(p)) return MAPLE_ERR_INVALID_ARG;
    for (const void *p : {(const void *)a.cu_q, (const void *)a.cu_k, (const void *)a.lse})
        if ((uintptr_t)p & 3u) return MAPLE_ERR_INVALID_ARG;
    for (int64_t s : {a.q_stride, a.k_stride, a.v_stride})
        if (s % 8 || s < 0 || s >= (1ll << 38)) return MAPLE_ERR_INVALID_ARG;
    PromptK k;
    k.a = a;
    k.G = a.heads / a.kv_heads;
    k.nt = 128 / k.G;
    if (k.a.window > (1 << 30)) k.a.window = 0;   // wider than any sequence
    CUtensorMap qm, km, vm;
    // (one row has no step to the next; without keys the maps stand on q and are not read)
    const int64_t qs = a.Tq > 1 ? a.q_stride : (int64_t)a.heads * D, own = (int64_t)a.kv_heads * D;
    int rc = head_map(&qm, a.q, a.dtype, a.Tq, a.heads, D, qs, k.G, k.nt);
    if (!rc) rc = head_map(&km, a.Tk ? a.k : a.q, a.dtype, a.Tk ? a.Tk : 1, a.kv_heads, D, a.Tk > 1 ? a.k_stride : own, 1, kKeys);
    if (!rc) rc = head_map(&vm, a.Tk ? a.v : a.q, a.dtype, a.Tk ? a.Tk : 1, a.kv_heads, D, a.Tk > 1 ? a.v_stride : own, 1, kKeys);
    if (rc) return rc;
    // no more pairs of tiles than this: every sequence rounds up once
    const int64_t span = 2 * k.nt, most = (a.max_q + span - 1) / span * a.B, all = a.Tq / span + a.B;
    const int64_t items = (most < all ? most : all) * a.kv_heads;
    if (items > 0x7fffffffll) return MAPLE_ERR_UNSUPPORTED_SHAPE;
    cudaStream_t st = (cudaStream_t)stream;
    if (a.dtype == MAPLE_BF16)
        return D == 128 ? launch<__nv_bfloat16, 128>(qm, km, vm, k, items, st) : launch<__nv_bfloat16, 64>(qm, km, vm, k, items, st);
    return D == 128 ? launch<__half, 128>(qm, km, vm, k, items, st) : launch<__half, 64>(qm, km, vm, k, items, st);
}
