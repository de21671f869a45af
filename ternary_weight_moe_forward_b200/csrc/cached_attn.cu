// Attention of one new token per sequence over the paged 4-bit cache.  C ABI:
// include/maple_attn.h.
//
// Mathematics.  For a group of 8 query heads that share a key/value head, the
// scores of 16 cached tokens are S^T = K Q^T (rows = tokens, columns = heads)
// and the output O^T += V^T P^T, both on m16n8k16 matrix instructions with the
// cached side as the 16-row operand, so that 8 heads fill an instruction.  A
// running maximum and sum per head make one pass over the cache enough.
//
// The 4-bit key codes c go into the matrix instructions as fp16 numbers, exactly:
// w & 0x000f000f is the pair (c, c') in units of fp16's smallest step, 2^-24, and
// with 0x00f000f0 it is 16 c, whose partner q is divided by 16.  With scale s and
// minimum m of a token's group of 32 channels,
//   q.k = 2^24 sum_groups s_g (q_g . c_g 2^-24) + sum_groups m_g sum(q_g)
// in 32 bits: the scores carry no rounding of the dequantised keys and no constant
// that cancels.  (As 1024 + c, with 1024 sum q taken off again, the partial sums
// were a hundred times the result and their last bits showed in peaked rows.)  q
// is brought to [1, 2) by a power of two per head first (exact), so that fp16
// holds it whatever its size.  Values are dequantised to fp16 (one rounding,
// 2^-11; 1024 + c less 1024 is exact there) and p, scaled by 2^4, is rounded to
// fp16 (bf16 outputs) or split in two fp16 terms (fp16 outputs, where one rounding
// of p would show).
//
// Work split.  All (sequence, key/value head) segments are laid end to end in
// units of 64 tokens and every CTA takes an equal share of the line, so that a
// batch of very different lengths keeps all SMs busy to the end.  A segment
// that lies in one CTA is finished there; a cut one leaves partial results (at
// most two per CTA) that combine_kernel joins in the order of the CTAs, so the
// result is the same every time.  Short bounds (a window) take one CTA per
// segment and no second kernel.
//
// Within a CTA each warp streams its own tiles of 64 tokens with bulk copies of
// whole pages, one tile ahead (one issuing thread per SM would not reach the
// memory's rate), and the warps' results are joined at a segment's end.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/maple_attn.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

using namespace maple;

namespace {

constexpr int kStages = 2, kTile = 64;   // tiles of a ring, tokens of a tile
constexpr int kCtas = 148;          // CTAs that share the line of all segments (one per SM)
constexpr int kSegCost = 12;        // tiles that a segment's own start and end are worth (64 ragged sequences: 4 104.7 us, 12 94.2, 24 95.6)
constexpr int kWholeTiles = 16;     // segments of at most so many tiles: one CTA each, no combine

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

struct CachedK {
    maple_attn_cached_args a;
    int NT, HB, cols;               // head tiles of 8, head blocks per key/value head, kv_heads * HB
    int whole;
    int64_t *prefix;                // [B] weight of the line before each sequence
    float *part_ml;                 // [2 kCtas][8 NT][2]
    float *part_o;                  // [2 kCtas][8 NT][D]
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with an accumulator of zeros
__device__ __forceinline__ void mma16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// (w & mask) | 0x64006400 in one instruction (written as two operators it became two)
template <uint32_t MASK>
__device__ __forceinline__ uint32_t codes(uint32_t w)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(MASK), "r"(0x64006400u));
    return r;
}
__device__ __forceinline__ uint32_t lo_codes(uint32_t w) { return codes<0x000f000fu>(w); }
__device__ __forceinline__ uint32_t hi_codes(uint32_t w) { return codes<0x00f000f0u>(w); }
__device__ __forceinline__ __half2 as_h2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }

// A sequence's tokens that its query sees, in tiles of 64
struct Span {
    int len, start, c0, n;
    __device__ __forceinline__ void load(const maple_attn_cached_args &a, int b)
    {
        const int64_t cap = (int64_t)a.max_pages * a.page_size;
        int64_t l = __ldg(a.lens + b);
        if (l > cap) l = cap;
        len = (int)l;
        start = a.window && len > a.window ? len - a.window : 0;
        c0 = start / kTile;
        n = len > 0 ? (len + kTile - 1) / kTile - c0 : 0;
    }
};

// How many CTAs share a line of `total` weight (tiles, and kSegCost for each segment): as few as leave each at most 8
// units, up to all of them.  A CTA whose share lies in segments' starts alone has no tile.
__device__ __forceinline__ int sharers(int64_t total) { return (int)min((int64_t)kCtas, (total + 7) / 8); }

// One warp per ring.  (In an earlier version two warps to a tile, 16 in all with
// 128 registers each, took 108 us where one took 96: what a tile costs beside its
// tokens was paid twice.)  16 heads leave room for 8 warps' accumulators.
template <int D, int NT>
struct CachedSmem {
    static constexpr int kWarps = NT == 1 ? 10 : 8, kHalf = (kWarps + 1) / 2;
    static constexpr int kTileBytes = kTile * KvPage<D>::kRowBytes;
    static constexpr int kBars = kWarps * kStages * kTileBytes;
    static constexpr int kOk = kBars + kWarps * kStages * 8;               // pages of each ring's tiles that hold tokens
    static constexpr int kMax = kOk + (kWarps * kStages * 4 + 15) / 16 * 16;                // [kWarps][16] maxima
    static constexpr int kSum = kMax + kWarps * 16 * 4;                    // [kHalf][16] sums
    static constexpr int kAcc = kSum + (kHalf * 16 * 4 + 15) / 16 * 16;    // [kHalf][NT][D / 16][32 lanes] float4
    static constexpr int kTotal = kAcc + kHalf * NT * (D / 16) * 512;
    static_assert(kAcc % 16 == 0, "the accumulators are moved as float4");
};

template <typename T, int D, int NT, int N>
__global__ void __launch_bounds__(CachedSmem<D, NT>::kWarps * 32, 1) cached_kernel(const CachedK p)
{
    using P = KvPage<D>;
    using L = CachedSmem<D, NT>;
    constexpr int kWarps = L::kWarps, KB = kTile / 16;   // blocks of 16 tokens in a tile
    constexpr int G = D / 32, MT = D / 16;     // groups of 32 channels, 16-channel tiles of V^T
    constexpr bool kSplitP = sizeof(T) == 2 && !__is_same(T, __nv_bfloat16);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[kWarps + 1];
    __shared__ int64_t s_first[2];
    __shared__ uint32_t s_abort;
    const maple_attn_cached_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int n = N, ppt = kTile / N;             // tokens of a page, pages of a tile
    constexpr int page_bytes = P::bytes(N);
    const uint32_t bar0 = smem_addr(smem + L::kBars) + warp * kStages * 8;
    volatile uint32_t *okmask = (volatile uint32_t *)(smem + L::kOk) + warp * kStages;
    if (lane == 0) {
        for (int s = 0; s < kStages; s++) mbar_init(bar0 + 8 * s, 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) s_abort = 0;
    volatile uint32_t *abort = &s_abort;

    // ---- this CTA's share of the line [R0, R1) and the segment that R0 falls into
    int64_t R0, R1, W;
    int b, col;
    if (p.whole) {
        b = blockIdx.x / p.cols;
        col = blockIdx.x - b * p.cols;
        W = R0 = 0;
        R1 = 1ll << 40;
        __syncthreads();
    } else {
        const int per = (a.B + blockDim.x - 1) / blockDim.x, lo = min((int)threadIdx.x * per, a.B), hi = min(lo + per, a.B);
        int64_t mine = 0;
        for (int i = lo; i < hi; i++) {
            Span s;
            s.load(a, i);
            mine += (int64_t)p.cols * (s.n + kSegCost);
        }
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int64_t before = inc - mine, total = 0;
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        const int ns = sharers(total);
        if ((int)blockIdx.x >= ns) return;
        R0 = total * blockIdx.x / ns;
        R1 = total * (blockIdx.x + 1) / ns;
        int64_t at = before;
        for (int i = lo; i < hi; i++) {
            Span s;
            s.load(a, i);
            const int64_t w = (int64_t)p.cols * (s.n + kSegCost);
            if (blockIdx.x == 0) p.prefix[i] = at;
            if (R0 >= at && R0 < at + w) {
                s_first[0] = i;
                s_first[1] = at;
            }
            at += w;
        }
        __syncthreads();
        b = (int)s_first[0];
        Span s;
        s.load(a, b);
        col = (int)((R0 - s_first[1]) / (s.n + kSegCost));
        W = s_first[1] + (int64_t)col * (s.n + kSegCost);
    }
    const int b_end = p.whole ? b + 1 : a.B;

    // ---- the ring's tiles, one after another over all segments of the share
    struct Walk {
        int b, col;
        int64_t W;
        Span s;
        int tile, end;      // next tile of this ring and the end of the share in the current segment
        int first, last;    // the share's tiles of this segment, counted from the segment's first
    };
    auto enter = [&](Walk &w) {
        w.first = (int)max(R0 - w.W - kSegCost, (int64_t)0);
        w.last = (int)min(max(R1 - w.W - kSegCost, (int64_t)0), (int64_t)w.s.n);
        w.tile = w.first + warp;
        w.end = w.last;
    };
    auto next_segment = [&](Walk &w) -> bool {
        w.W += w.s.n + kSegCost;
        if (++w.col == p.cols || p.whole) {
            w.col = 0;
            if (++w.b >= b_end) return false;
            w.s.load(a, w.b);
        }
        if (w.W >= R1) return false;
        enter(w);
        return true;
    };

    Walk pf;
    pf.b = b;
    pf.col = col;
    pf.W = W;
    pf.s.load(a, b);
    enter(pf);
    Walk cur = pf;
    bool have = true;
    int page = -1;              // lane i: page of the candidate's i-th page, loaded one step ahead of its copy
    bool wanted = false;
    auto settle = [&]() {       // to the next tile of this ring, and its pages' numbers on their way
        while (have && pf.tile >= pf.end) have = next_segment(pf);
        page = -1;
        wanted = false;
        if (have && lane < ppt) {
            const int j0 = (pf.s.c0 + pf.tile) * kTile + lane * n;
            wanted = j0 < pf.s.len && j0 + n > pf.s.start;
            if (wanted) page = __ldg(a.block_table + (int64_t)pf.b * a.table_stride + j0 / n);
        }
    };
    auto issue = [&](int s) {
        if (have) {
            const bool good = wanted && page >= 0 && page < a.num_pages;
            if (wanted && !good) set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
            const uint32_t m = __ballot_sync(FULL, good);
            if (lane == 0) okmask[s] = m;   // (read after the wait on the barrier and a warp barrier)
            const uint32_t bar = bar0 + 8 * s;
            if (lane == 0) {
                if (m) mbar_expect_tx(bar, __popc(m) * page_bytes);
                else mbar_arrive(bar);
            }
            __syncwarp();
            if (good)
                bulk_g2s(smem_addr(smem + (warp * kStages + s) * L::kTileBytes + lane * page_bytes),
                         a.pages + ((int64_t)page * a.kv_heads + pf.col / p.HB) * page_bytes, page_bytes, bar);
            pf.tile += kWarps;
            settle();
        }
    };
    uint32_t issued = 0, used = 0;   // tiles of this ring
    settle();
    for (int s = 0; s < kStages; s++) {
        if (have) issued++;
        issue(s);
    }

    const int heads_per = a.heads / a.kv_heads;
    bool dead = false;
    for (bool more = true; more;) {
        const int kvh = cur.col / p.HB, h0 = (cur.col - kvh * p.HB) * 8 * NT;
        const int nh = min(8 * NT, heads_per - h0);              // heads of this block
        const int ntile = cur.last - cur.first;
        const bool empty = cur.s.n == 0 && R0 <= cur.W;          // no tokens: the share that holds its start writes zeros
        if (R0 <= cur.W && threadIdx.x == 0 && __ldg(a.lens + cur.b) > (int64_t)a.max_pages * n)
            set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
        if (ntile > 0 || empty) {
            // ---- queries: B fragments, their sums, and the softmax scale of this lane's two heads
            uint32_t qf[NT][G][4];
            uint32_t qs[NT][2];
            float sc[NT][2];
#pragma unroll
            for (int j = 0; j < NT; j++) {
                const int h = j * 8 + g;
                uint4 raw[G];
#pragma unroll
                for (int i = 0; i < G; i++) raw[i] = make_uint4(0, 0, 0, 0);
                if (h < nh && ntile > 0) {
                    const T *src = (const T *)a.q + (int64_t)cur.b * a.q_stride + (int64_t)(kvh * heads_per + h0 + h) * D + 8 * t;
#pragma unroll
                    for (int i = 0; i < G; i++) raw[i] = __ldg(reinterpret_cast<const uint4 *>(src + 32 * i));
                }
                qs[j][0] = qs[j][1] = 0;
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < G; i++) {
                    float x[8];
                    unpack8<T>(raw[i], x);
#pragma unroll
                    for (int m = 0; m < 8; m++) amax = fmaxf(amax, fabsf(x[m]));
                }
                amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 2));
                // 2^-e with amax * 2^-e in [1, 2) (as far as 2^-e and 2^e are normal); 1 for zero and what is not finite
                int e = (int)(__float_as_uint(amax) >> 23) - 127;
                if (e >= 127 || e < -120) e = e == 127 ? 126 : (amax == 0.0f || e == 128 ? 0 : -120);
                const float down = copysignf(__int_as_float((127 - e) << 23), a.scale);
                // (a negative scale goes into q; 10^-30 is as good as 0 and keeps -inf * scale)
                const float mine_sc = fmaxf(fabsf(a.scale) * 1.4426950408889634f * __int_as_float((127 + e) << 23), 1e-30f);
#pragma unroll
                for (int i = 0; i < G; i++) {
                    float x[8];
                    unpack8<T>(raw[i], x);
#pragma unroll
                    for (int m = 0; m < 8; m++) x[m] = x[m] * down * ((m & 1) ? 0.0625f : 1.0f);
                    float sum = 0.0f;
#pragma unroll
                    for (int m = 0; m < 4; m++) {
                        const __half2 v = __floats2half2_rn(x[m], x[m + 4]);
                        qf[j][i][m] = as_u32(v);
                        const float2 f = __half22float2(v);
                        sum += (m & 1) ? 16.0f * (f.x + f.y) : f.x + f.y;
                    }
                    sum += __shfl_xor_sync(FULL, sum, 1);
                    sum += __shfl_xor_sync(FULL, sum, 2);
                    if (i == t) {   // rows 2t+1 (the minima of group t) in two fp16 terms, 22 bits
                        const __half hi = __float2half_rn(sum);
                        const __half2 h2 = __halves2half2(__float2half_rn(0.0f), hi);
                        const __half2 l2 = __halves2half2(__float2half_rn(0.0f), __float2half_rn(sum - __half2float(hi)));
                        qs[j][0] = as_u32(h2);
                        qs[j][1] = as_u32(l2);
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; c++) sc[j][c] = __shfl_sync(FULL, mine_sc, (2 * t + c) * 4);
            }
            float O[NT][MT][4], mx[NT][2], sum[NT][2];
#pragma unroll
            for (int j = 0; j < NT; j++) {
#pragma unroll
                for (int i = 0; i < MT; i++)
#pragma unroll
                    for (int c = 0; c < 4; c++) O[j][i][c] = 0.0f;
                mx[j][0] = mx[j][1] = -INFINITY;
                sum[j][0] = sum[j][1] = 0.0f;
            }

            // ---- this ring's tiles of the segment
            for (int tile = cur.first + warp; tile < cur.last; tile += kWarps) {
                const int s = used % kStages;
                if (!dead && !mbar_wait(bar0 + 8 * s, (used / kStages) & 1, abort, a.flags, kDefaultWaitNs)) dead = true;
                dead = __any_sync(FULL, dead);
                const uint8_t *buf = smem + (warp * kStages + s) * L::kTileBytes;
                const uint32_t ok = okmask[s];
                const int j0 = (cur.s.c0 + tile) * kTile;
                const bool edge = j0 < cur.s.start || j0 + kTile > cur.s.len || ok != (1u << ppt) - 1;
                if (!dead) {
                    float S[NT][KB][4];
#pragma unroll
                    for (int kb = 0; kb < KB; kb++) {
                        const int k0 = kb * 16, pg = k0 / n, r0 = k0 % n;
                        const uint8_t *base = buf + pg * page_bytes;
                        uint32_t w0[G], w1[G], pr0[G], pr1[G];
                        if (G == 4) {
                            *(uint4 *)w0 = *(const uint4 *)(base + (r0 + g) * (D / 2) + t * 16);
                            *(uint4 *)w1 = *(const uint4 *)(base + (r0 + g + 8) * (D / 2) + t * 16);
                            *(uint4 *)pr0 = *(const uint4 *)(base + P::k_pair(n, r0 + g, 0));
                            *(uint4 *)pr1 = *(const uint4 *)(base + P::k_pair(n, r0 + g + 8, 0));
                        } else {
                            *(uint2 *)w0 = *(const uint2 *)(base + (r0 + g) * (D / 2) + t * 8);
                            *(uint2 *)w1 = *(const uint2 *)(base + (r0 + g + 8) * (D / 2) + t * 8);
                            *(uint2 *)pr0 = *(const uint2 *)(base + P::k_pair(n, r0 + g, 0));
                            *(uint2 *)pr1 = *(const uint2 *)(base + P::k_pair(n, r0 + g + 8, 0));
                        }
                        // sum_groups m_g sum(q_g): the (scale, minimum) pairs themselves as the 16-row operand
                        const uint32_t mp0 = *(const uint32_t *)(base + P::k_pair(n, r0 + g, t % G));
                        const uint32_t mp1 = *(const uint32_t *)(base + P::k_pair(n, r0 + g + 8, t % G));
                        float sum_c[NT][4];      // sum_groups s_g (q_g . c_g), in units of 2^-24
#pragma unroll
                        for (int i = 0; i < G; i++) {
                            const uint32_t x0 = w0[i] >> 8, x1 = w1[i] >> 8;
                            const uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
                            const float s0 = __low2float(as_h2(pr0[i])), s1 = __low2float(as_h2(pr1[i]));
#pragma unroll
                            for (int j = 0; j < NT; j++) {
                                float c[4];
                                mma16_zero(c, w0[i] & lo, w1[i] & lo, w0[i] & hi, w1[i] & hi, qf[j][i][0], qf[j][i][1]);
                                mma16(c, x0 & lo, x1 & lo, x0 & hi, x1 & hi, qf[j][i][2], qf[j][i][3]);
#pragma unroll
                                for (int e = 0; e < 4; e++) {
                                    const float se = e < 2 ? s0 : s1;
                                    sum_c[j][e] = i == 0 ? se * c[e] : fmaf(se, c[e], sum_c[j][e]);
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < NT; j++) {
                            mma16_zero(S[j][kb], mp0, mp1, mp0, mp1, qs[j][0], qs[j][1]);
#pragma unroll
                            for (int e = 0; e < 4; e++) S[j][kb][e] = fmaf(sum_c[j][e], 16777216.0f, S[j][kb][e]);
                        }
                        if (edge) {
                            const bool okp = (ok >> pg) & 1;
#pragma unroll
                            for (int half = 0; half < 2; half++) {
                                const int key = j0 + k0 + g + 8 * half;
                                if (!okp || key < cur.s.start || key >= cur.s.len) {
#pragma unroll
                                    for (int j = 0; j < NT; j++) S[j][kb][2 * half] = S[j][kb][2 * half + 1] = -INFINITY;
                                }
                            }
                        }
                    }
                    // ---- weights 2^(score - reference + 4).  The reference follows the maximum only when a
                    // score passes it by 2^8 (fp16 holds 2^12), which a vote finds without reducing over the
                    // lanes; the sums do not depend on it otherwise.
#pragma unroll
                    for (int j = 0; j < NT; j++) {
                        float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int kb = 0; kb < KB; kb++)
#pragma unroll
                            for (int c = 0; c < 4; c++) m[c & 1] = fmaxf(m[c & 1], S[j][kb][c]);
                        const bool above = m[0] * sc[j][0] > mx[j][0] + 8.0f || m[1] * sc[j][1] > mx[j][1] + 8.0f;
                        if (__any_sync(FULL, above)) {
                            float f[2];
#pragma unroll
                            for (int c = 0; c < 2; c++) {
                                float v = m[c] * sc[j][c];
                                v = fmaxf(v, __shfl_xor_sync(FULL, v, 4));
                                v = fmaxf(v, __shfl_xor_sync(FULL, v, 8));
                                v = fmaxf(v, __shfl_xor_sync(FULL, v, 16));
                                v = fmaxf(mx[j][c], v);
                                f[c] = mx[j][c] == -INFINITY ? 0.0f : ex2(mx[j][c] - v);
                                sum[j][c] *= f[c];
                                mx[j][c] = v;
                            }
#pragma unroll
                            for (int i = 0; i < MT; i++) {
                                O[j][i][0] *= f[0];
                                O[j][i][1] *= f[1];
                                O[j][i][2] *= f[0];
                                O[j][i][3] *= f[1];
                            }
                        }
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            const float off = mx[j][c] == -INFINITY ? 0.0f : 4.0f - mx[j][c];
#pragma unroll
                            for (int kb = 0; kb < KB; kb++)
#pragma unroll
                                for (int half = 0; half < 2; half++) {
                                    float &v = S[j][kb][2 * half + c];
                                    v = ex2(fmaf(v, sc[j][c], off));
                                    sum[j][c] += v;
                                }
                        }
                    }
                    // ---- O^T += V^T P^T
#pragma unroll
                    for (int kb = 0; kb < KB; kb++) {
                        const int k0 = kb * 16, pg = k0 / n, r0 = k0 % n;
                        const uint8_t *base = buf + pg * page_bytes;
                        const uint8_t *vb = base + n * (D / 2) + (r0 >> 4) * (8 * D) + lane * 16;
                        const int gg = g * (D / 8) / 32;   // the group of this lane's channels
                        // scales and minima of tokens (2t, 2t+1) and (2t+8, 2t+9)
                        uint32_t s0 = *(const uint32_t *)(base + P::v_scale(n, r0 + 2 * t, gg));
                        uint32_t s1 = *(const uint32_t *)(base + P::v_scale(n, r0 + 2 * t + 8, gg));
                        uint32_t m0 = *(const uint32_t *)(base + P::v_min(n, r0 + 2 * t, gg));
                        uint32_t m1 = *(const uint32_t *)(base + P::v_min(n, r0 + 2 * t + 8, gg));
                        if (edge) {   // rows without a token may hold anything: their weight is 0, their value too
                            const bool okp = (ok >> pg) & 1;
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const int key = j0 + k0 + 2 * t + (i & 1) + 8 * (i >> 1);
                                if (!okp || key < cur.s.start || key >= cur.s.len) {
                                    const uint32_t keep = (i & 1) ? 0x0000ffffu : 0xffff0000u;
                                    if (i < 2) { s0 &= keep; m0 &= keep; }
                                    else { s1 &= keep; m1 &= keep; }
                                }
                            }
                        }
                        uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
                        for (int j = 0; j < NT; j++)
#pragma unroll
                            for (int half = 0; half < 2; half++) {
                                const float v0 = S[j][kb][2 * half], v1 = S[j][kb][2 * half + 1];
                                const __half2 hi = __floats2half2_rn(v0, v1);
                                pb[j][half] = transpose8(as_u32(hi));
                                if (kSplitP) {
                                    const float2 f = __half22float2(hi);
                                    pl[j][half] = transpose8(as_u32(__floats2half2_rn(v0 - f.x, v1 - f.y)));
                                }
                            }
                        const __half2 k1024 = __float2half2_rn(-1024.0f), k64 = __float2half2_rn(-64.0f), k16 = __float2half2_rn(0.0625f);
                        auto deq_lo = [&](uint32_t w, uint32_t s, uint32_t m) {
                            return as_u32(__hfma2(__hadd2(as_h2(lo_codes(w)), k1024), as_h2(s), as_h2(m)));
                        };
                        auto deq_hi = [&](uint32_t w, uint32_t s, uint32_t m) {
                            return as_u32(__hfma2(__hfma2(as_h2(hi_codes(w)), k16, k64), as_h2(s), as_h2(m)));
                        };
                        uint4 va = *(const uint4 *)vb, vc = va;
                        if (D == 128) vc = *(const uint4 *)(vb + 512);
                        // words of tokens 2t, 2t+1 (e, o) and 2t+8, 2t+9 (e8, o8)
                        constexpr int NW = D / 64;
                        const uint32_t e[2] = {va.x, va.y}, o[2] = {D == 128 ? va.z : va.y, va.w};
                        const uint32_t e8[2] = {D == 128 ? vc.x : vc.z, vc.y}, o8[2] = {D == 128 ? vc.z : vc.w, vc.w};
#pragma unroll
                        for (int w = 0; w < NW; w++)
#pragma unroll
                            for (int q = 0; q < 2; q++) {   // channels 4q .. 4q+3 of the word
                                uint32_t x = __byte_perm(e[w], o[w], q ? 0x7632 : 0x5410);
                                uint32_t y = __byte_perm(e8[w], o8[w], q ? 0x7632 : 0x5410);
#pragma unroll
                                for (int z = 0; z < 2; z++) {
                                    const uint32_t a0 = deq_lo(x, s0, m0), a1 = deq_hi(x, s0, m0);
                                    const uint32_t a2 = deq_lo(y, s1, m1), a3 = deq_hi(y, s1, m1);
#pragma unroll
                                    for (int j = 0; j < NT; j++) {
                                        mma16(O[j][w * 4 + q * 2 + z], a0, a1, a2, a3, pb[j][0], pb[j][1]);
                                        if (kSplitP) mma16(O[j][w * 4 + q * 2 + z], a0, a1, a2, a3, pl[j][0], pl[j][1]);
                                    }
                                    x >>= 8;
                                    y >>= 8;
                                }
                            }
                    }
                }
                __syncwarp();     // the tile is read
                used++;
                if (have) issued++;
                issue(s);
            }

            // ---- join the warps: common maximum, then sums in a fixed tree
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    sum[j][c] += __shfl_xor_sync(FULL, sum[j][c], 4);
                    sum[j][c] += __shfl_xor_sync(FULL, sum[j][c], 8);
                    sum[j][c] += __shfl_xor_sync(FULL, sum[j][c], 16);
                }
            float *s_max = (float *)(smem + L::kMax), *s_sum = (float *)(smem + L::kSum);
            float4 *s_acc = (float4 *)(smem + L::kAcc);
            if (g == 0)
#pragma unroll
                for (int j = 0; j < NT; j++)
#pragma unroll
                    for (int c = 0; c < 2; c++) s_max[warp * 16 + j * 8 + 2 * t + c] = mx[j][c];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NT; j++) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    float m = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; w++) m = fmaxf(m, s_max[w * 16 + j * 8 + 2 * t + c]);
                    f[c] = mx[j][c] == -INFINITY ? 0.0f : ex2(mx[j][c] - m);
                    mx[j][c] = m;
                    sum[j][c] *= f[c];
                }
#pragma unroll
                for (int i = 0; i < MT; i++) {
                    O[j][i][0] *= f[0];
                    O[j][i][1] *= f[1];
                    O[j][i][2] *= f[0];
                    O[j][i][3] *= f[1];
                }
            }
            const int busy = min(kWarps, ntile);    // (warps beyond the tiles hold zeros)
            if (busy <= 1) __syncthreads();         // the maxima are read before the next segment's are written
            for (int m = busy; m > 1;) {
                const int half = (m + 1) / 2;
                if (warp >= half && warp < m) {
#pragma unroll
                    for (int j = 0; j < NT; j++) {
#pragma unroll
                        for (int i = 0; i < MT; i++)
                            s_acc[(((warp - half) * NT + j) * MT + i) * 32 + lane] =
                                make_float4(O[j][i][0], O[j][i][1], O[j][i][2], O[j][i][3]);
                        if (g == 0) {
                            s_sum[(warp - half) * 16 + j * 8 + 2 * t] = sum[j][0];
                            s_sum[(warp - half) * 16 + j * 8 + 2 * t + 1] = sum[j][1];
                        }
                    }
                }
                __syncthreads();
                if (warp < m - half) {
#pragma unroll
                    for (int j = 0; j < NT; j++) {
#pragma unroll
                        for (int i = 0; i < MT; i++) {
                            const float4 v = s_acc[((warp * NT + j) * MT + i) * 32 + lane];
                            O[j][i][0] += v.x;
                            O[j][i][1] += v.y;
                            O[j][i][2] += v.z;
                            O[j][i][3] += v.w;
                        }
                        sum[j][0] += s_sum[warp * 16 + j * 8 + 2 * t];
                        sum[j][1] += s_sum[warp * 16 + j * 8 + 2 * t + 1];
                    }
                }
                __syncthreads();
                m = half;
            }
            // ---- warp 0 holds the segment's (or the share's) result
            if (warp == 0) {
                const bool whole_seg = cur.first == 0 && cur.last == cur.s.n;
                const int slot = 2 * blockIdx.x + (R0 >= cur.W ? 0 : 1);
                constexpr int CH = D / 8;          // channels of this lane, CH*g ..
#pragma unroll
                for (int j = 0; j < NT; j++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        const int h = j * 8 + 2 * t + c;
                        if (h >= nh) continue;
                        float x[CH];
#pragma unroll
                        for (int i = 0; i < MT; i++) {
                            x[2 * i] = O[j][i][c];
                            x[2 * i + 1] = O[j][i][c + 2];
                        }
                        if (whole_seg) {
                            const float inv = sum[j][c] > 0.0f || sum[j][c] != sum[j][c] ? __fdiv_rn(1.0f, sum[j][c]) : 0.0f;
                            T *dst = (T *)a.out + ((int64_t)cur.b * a.heads + kvh * heads_per + h0 + h) * D + CH * g;
#pragma unroll
                            for (int i = 0; i < CH; i += 8) {
                                float y[8];
#pragma unroll
                                for (int m = 0; m < 8; m++) y[m] = x[i + m] * inv;
                                *reinterpret_cast<uint4 *>(dst + i) = pack8<T>(y);
                            }
                        } else {
                            float *dst = p.part_o + ((int64_t)slot * 8 * NT + h) * D + CH * g;
#pragma unroll
                            for (int i = 0; i < CH; i += 4)
                                *reinterpret_cast<float4 *>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                            if (g == 0) {
                                p.part_ml[((int64_t)slot * 8 * NT + h) * 2] = mx[j][c];
                                p.part_ml[((int64_t)slot * 8 * NT + h) * 2 + 1] = sum[j][c];
                            }
                        }
                    }
            }
        }
        more = next_segment(cur);
    }
    for (; used < issued; used++)   // copies still in flight (only after a failed wait)
        mbar_wait(bar0 + 8 * (used % kStages), (used / kStages) & 1, abort, a.flags, kDefaultWaitNs);
    asm volatile("griddepcontrol.launch_dependents;");
}

// Joins the partial results of segments that several CTAs share: one CTA per
// (sequence, column, head), its 8 warps taking every eighth partial result and
// summed in order, so that all loads are in flight at once (a loop over the
// partial results by one thread per output cost 40 us for 75 of them).  A warp's
// first kEarly partial results are loaded before their factors are known: one
// sequence of 131071 tokens took 22.6 us in all instead of 26.5.  Ten for each of 8
// warps hold the 74 or 75 that one sequence over two key/value heads leaves (six:
// 22.9 to 23.7 us against 22.5); more, up to 148 with one key/value head, go through
// the loop behind them.  They cost a ragged batch, which has few, 0.3 of 94.2 us.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(256, 4) combine_kernel(const CachedK p)
{
    constexpr int V = D / 32, kEarly = 10;      // channels of a lane, partial results loaded before their factors are known
    __shared__ float s_f[kCtas], s_l[8], s_acc[8][D], s_m[8];
    const maple_attn_cached_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / p.cols, col = blockIdx.x - b * p.cols, h = blockIdx.y;
    const int heads_per = a.heads / a.kv_heads, kvh = col / p.HB, h0 = (col - kvh * p.HB) * 8 * NT;
    Span s, e;
    s.load(a, b);
    e.load(a, a.B - 1);
    // Every block waits (the lengths are not cached_kernel's, they are read before): if all of them could return
    // first, as for a batch without a token, what follows this kernel would not be ordered behind cached_kernel.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (s.n == 0 || h >= heads_per - h0) return;
    const int64_t total = p.prefix[a.B - 1] + (int64_t)p.cols * (e.n + kSegCost);
    const int ns = sharers(total);
    const int64_t W = p.prefix[b] + (int64_t)col * (s.n + kSegCost);
    // the share that holds position x of the line: the largest i with total * i / ns <= x
    auto share = [&](int64_t x) { return (int)(((x + 1) * ns - 1) / total); };
    const int i0 = share(W + kSegCost), i1 = share(W + kSegCost + s.n - 1);
    if (i0 == i1) return;
    const int first_slot = 2 * i0 + (total * i0 / ns >= W ? 0 : 1);   // (later shares begin inside the segment)
    auto at = [&](int i) { return (int64_t)(i == i0 ? first_slot : 2 * i) * 8 * NT + h; };
    const int np = i1 - i0 + 1;
    // the first partial results of the warp, on their way under the factors
    auto fetch = [&](int i, float (&x)[V]) {
        const float *src = p.part_o + at(i0 + i) * D + V * lane;
        if (V == 4) *(float4 *)x = *reinterpret_cast<const float4 *>(src);
        else *(float2 *)x = *reinterpret_cast<const float2 *>(src);
    };
    float early[kEarly][V];
#pragma unroll
    for (int j = 0; j < kEarly; j++)
        if (warp + 8 * j < np) fetch(warp + 8 * j, early[j]);
    // factors of the partial results
    float2 ml = make_float2(-INFINITY, 0.0f);
    if ((int)threadIdx.x < np) ml = *reinterpret_cast<const float2 *>(p.part_ml + at(i0 + threadIdx.x) * 2);
    const float wm = warp_max(ml.x);
    if (lane == 0) s_m[warp] = wm;
    __syncthreads();
    float m = s_m[0];
#pragma unroll
    for (int w = 1; w < 8; w++) m = fmaxf(m, s_m[w]);
    const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
    if ((int)threadIdx.x < np) s_f[threadIdx.x] = f;
    const float wl = warp_tree_sum(f * ml.y);
    if (lane == 0) s_l[warp] = wl;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; v++) acc[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < kEarly; j++)
        if (warp + 8 * j < np) {
            const float fi = s_f[warp + 8 * j];
#pragma unroll
            for (int v = 0; v < V; v++) acc[v] = fmaf(early[j][v], fi, acc[v]);
        }
#pragma unroll 5
    for (int i = warp + 8 * kEarly; i < np; i += 8) {
        const float fi = s_f[i];
        float x[V];
        fetch(i, x);
#pragma unroll
        for (int v = 0; v < V; v++) acc[v] = fmaf(x[v], fi, acc[v]);
    }
#pragma unroll
    for (int v = 0; v < V; v++) s_acc[warp][V * lane + v] = acc[v];
    __syncthreads();
    if (threadIdx.x < D / 2) {
        float l = 0.0f, x0 = 0.0f, x1 = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; w++) {
            l += s_l[w];
            x0 += s_acc[w][2 * threadIdx.x];
            x1 += s_acc[w][2 * threadIdx.x + 1];
        }
        const float inv = l > 0.0f || l != l ? __fdiv_rn(1.0f, l) : 0.0f;
        reinterpret_cast<uint32_t *>((T *)a.out + ((int64_t)b * a.heads + kvh * heads_per + h0 + h) * D)[threadIdx.x] =
            Elem<T>::pack(x0 * inv, x1 * inv);
    }
}

// the plan that the workspace and the launch share
struct Plan {
    int NT, HB, cols, whole;
    int64_t prefix_bytes, ml_bytes, o_bytes;
};
Plan make_plan(int32_t B, int32_t max_pages, int32_t heads, int32_t kv_heads, int32_t D, int32_t page_size, int32_t window)
{
    Plan pl;
    const int G = heads / kv_heads;
    pl.NT = G <= 8 ? 1 : 2;
    pl.HB = (G + 8 * pl.NT - 1) / (8 * pl.NT);
    pl.cols = kv_heads * pl.HB;
    int64_t tokens = (int64_t)max_pages * page_size;
    if (window && tokens > (int64_t)window + kTile - 1) tokens = (int64_t)window + kTile - 1;
    pl.whole = (tokens + kTile - 1) / kTile <= kWholeTiles;
    pl.prefix_bytes = pl.whole ? 0 : ((int64_t)B * 8 + 255) / 256 * 256;
    pl.ml_bytes = pl.whole ? 0 : (2ll * kCtas * 8 * pl.NT * 8 + 255) / 256 * 256;
    pl.o_bytes = pl.whole ? 0 : 2ll * kCtas * 8 * pl.NT * D * 4;
    return pl;
}

template <typename T, int D, int NT>
int launch(const CachedK &k, cudaStream_t st)
{
    const int smem = CachedSmem<D, NT>::kTotal;
    auto kernel = k.a.page_size == 16   ? cached_kernel<T, D, NT, 16>
                  : k.a.page_size == 32 ? cached_kernel<T, D, NT, 32>
                                        : cached_kernel<T, D, NT, 64>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return MAPLE_ERR_CUDA;
    }
    const int64_t segments = (int64_t)k.a.B * k.cols;
    kernel<<<(unsigned)(k.whole ? segments : kCtas), CachedSmem<D, NT>::kWarps * 32, smem, st>>>(k);
    if (!k.whole) {
        cudaLaunchConfig_t lc;
        memset(&lc, 0, sizeof lc);
        lc.gridDim = dim3((unsigned)segments, 8 * NT);
        lc.blockDim = dim3(256);
        lc.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        if (cudaLaunchKernelEx(&lc, combine_kernel<T, D, NT>, k) != cudaSuccess) {
            cudaGetLastError();
            return MAPLE_ERR_CUDA;
        }
    }
    return cudaGetLastError() == cudaSuccess ? MAPLE_OK : MAPLE_ERR_CUDA;
}

template <typename T>
int launch_type(const CachedK &k, cudaStream_t st)
{
    if (k.a.head_dim == 128) return k.NT == 1 ? launch<T, 128, 1>(k, st) : launch<T, 128, 2>(k, st);
    return k.NT == 1 ? launch<T, 64, 1>(k, st) : launch<T, 64, 2>(k, st);
}

}  // namespace

extern "C" int64_t maple_attn_cached_workspace(int32_t B, int32_t max_pages, int32_t heads, int32_t kv_heads,
                                               int32_t head_dim, int32_t page_size, int32_t window)
{
    if (maple_attn_page_bytes(head_dim, page_size) < 0 || heads < 1 || kv_heads < 1 || heads > 1024 || heads % kv_heads)
        return MAPLE_ERR_UNSUPPORTED_SHAPE;
    if (B < 0 || B > 65535 || max_pages < 0 || max_pages > (1 << 30) / page_size || window < 0) return MAPLE_ERR_INVALID_ARG;
    const Plan pl = make_plan(B, max_pages, heads, kv_heads, head_dim, page_size, window);
    return pl.prefix_bytes + pl.ml_bytes + pl.o_bytes;
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
    const Plan pl = make_plan(a.B, a.max_pages, a.heads, a.kv_heads, a.head_dim, a.page_size, a.window);
    CachedK k;
    k.a = a;
    k.NT = pl.NT;
    k.HB = pl.HB;
    k.cols = pl.cols;
    k.whole = pl.whole;
    k.prefix = (int64_t *)a.workspace;
    k.part_ml = (float *)((char *)a.workspace + pl.prefix_bytes);
    k.part_o = (float *)((char *)a.workspace + pl.prefix_bytes + pl.ml_bytes);
    return a.dtype == MAPLE_BF16 ? launch_type<__nv_bfloat16>(k, (cudaStream_t)stream) : launch_type<__half>(k, (cudaStream_t)stream);
}
