// Causal attention over packed prompts on the 5th-generation tensor cores.
// C ABI: include/maple_attn.h.
//
// Mathematics.  S = Q K^T and O += P V on tcgen05 (kind::f16, M = 128, fp32
// accumulators in tensor memory), P = 2^(scale2 S - m) with a running reference
// m per row and the row sum l beside it, out = O / l.  The reference follows
// the row maximum only when a score passes it by 2^8: until then P stays below
// 256, the sums stay exact in the same way, and O need not be rescaled.  P is
// rounded to the inputs' type (the tensor cores' operand); l sums it before the
// rounding.  For fp16 heads P carries a factor of 2^7 (at most 2^15 then, fp16
// ends at 2^16), which cancels in O / l: fp16's smallest step, 2^-24, is 2^-31 of
// the reference so, and many weights far below the largest keep their share.
//
// Rows.  A tile is 128 rows = floor(128/G) query tokens x the G query heads of
// one key/value head, so that grouped heads share every K and V tile (one 3-D
// TMA box brings them, whatever G), and a short prompt fills a tile with heads.
//
// One CTA works on two tiles (A and B, consecutive tokens) of a sequence and a
// key/value head, over tiles of 128 keys:
//   warps 0-3 softmax of A, warps 4-7 of B: one thread per row, S from tensor
//             memory, P back; rescaling and the epilogue
//   warp 8    TMA: Q once, then pairs (K_j, V_j-1) into a ring
//   warp 9    MMA, per pair: S = Q_A K_j, O_A += P_A V_j-1, the same for B
//   warp 10   the CTA's items, one ahead: the loads and first products of the
//             next item run under the last softmax and epilogue of this one
// While one tile's rows are in the exponentials, the tensor cores work on the
// other's products and on this one's next scores: tensor memory holds one S that
// A and B use in turn (it is free again as soon as its rows are in registers),
// P_A, P_B, O_A and O_B: 512 columns at d = 128.
//
// Masked keys.  P is 0 there, but 0 times an infinity or NaN in V would reach
// the sums; so tiles that hold masked keys have what is not finite in V set to
// 0 in shared memory first, and if anything was found the rows that do see
// those values add them again at the end.
//
// Work is ordered from the last tokens (the longest rows) to the first, so that
// the short items fill the end of the run; CTAs that are done take over blocks
// that have not started (cluster launch control).
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
template <typename T>
constexpr float kLift = __is_same(T, __half) ? 7.0f : 0.0f;   // P carries a factor of 2^kLift

template <int D>
struct PromptSmem {
    static constexpr int kHalves = D / 64;                 // 64-column (128-byte) sub-tiles
    static constexpr int kTileBytes = kHalves * 128 * 128; // a Q, K or V tile
    static constexpr int kStages = D == 128 ? 2 : 4;       // pairs of a ring: K_j in the first half, V_j-1 in the second
    static constexpr int kKv = 2 * kTileBytes;             // after Q_A and Q_B
    static constexpr int kBars = kKv + kStages * 2 * kTileBytes;
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

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// the largest of three
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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

// one lane of the warp, the same every time
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// the bits of the two 16-bit halves of w that hold an infinity or NaN
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t E = sizeof(T) && __is_same(T, __nv_bfloat16) ? 0x7f80u : 0x7c00u;
    return ((w & E) == E ? 0xffffu : 0u) | ((w & (E << 16)) == (E << 16) ? 0xffff0000u : 0u);
}

// Cluster launch control: a running CTA takes over one that has not started, so
// that items are handed out as CTAs get free, without a counter in memory.
__device__ __forceinline__ void try_cancel(uint32_t dst, uint32_t bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ int cancelled_block(const uint4 *resp)   // its blockIdx.x, or -1
{
    int x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b64 lo, hi;\n\t"
        "ld.shared.v2.b64 {lo, hi}, [%1];\n\t"
        "mov.b128 r, {lo, hi};\n\t"
        "mov.s32 %0, -1;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
        : "=r"(x)
        : "r"(smem_addr(resp))
        : "memory");
    return x;
}

// An item: a pair of tiles of one sequence and key/value head
struct Item {
    int kvh, tA, q0, lq, k0, off;      // kvh < 0: no more
};

// The item of a block: (sequence, pair) in the order of the sequences from the
// last one, a sequence's pairs from its last tokens, key/value heads fastest.
// One warp; 32 sequences at a time, or 256 (8 per lane) where there are more than
// 32.  kvh = -2: beyond the last item.
__device__ __forceinline__ Item find_item(const maple_attn_prompt_args &a, int nt, int block)
{
    const int lane = threadIdx.x & 31, span = 2 * nt;
    Item it;
    it.kvh = -2;
    const int x = block / a.kv_heads;
    auto rows = [&](int b, int64_t &q0, int64_t &q1) {      // query rows, as cut to Tq
        q0 = min(max((int64_t)__ldg(a.cu_q + b), (int64_t)0), a.Tq);
        q1 = min(max((int64_t)__ldg(a.cu_q + b + 1), q0), a.Tq);
    };
    auto pairs = [&](int b) {
        int64_t q0, q1;
        rows(b, q0, q1);
        return (int)((min(q1 - q0, (int64_t)a.max_q) + span - 1) / span);
    };
    const int per = a.B > 32 ? 8 : 1;
    int at = 0;
    for (int b0 = a.B - 1; b0 >= 0; b0 -= 32 * per) {
        int sum = 0;
        for (int i = 0; i < per; i++)
            if (b0 - lane * per - i >= 0) sum += pairs(b0 - lane * per - i);
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += v;
        }
        const unsigned hit = __ballot_sync(FULL, x >= at + inc - sum && x < at + inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            int b = b0 - src * per, rest = x - __shfl_sync(FULL, at + inc - sum, src), n;
            while (rest >= (n = pairs(b))) {
                rest -= n;
                b--;
            }
            int64_t q0, q1;
            rows(b, q0, q1);
            const int64_t k0 = min(max((int64_t)__ldg(a.cu_k + b), (int64_t)0), a.Tk);
            const int64_t k1 = min(max((int64_t)__ldg(a.cu_k + b + 1), k0), a.Tk);
            it.kvh = block - x * a.kv_heads;
            it.tA = (n - 1 - rest) * span;
            it.q0 = (int)q0;
            it.lq = (int)min(q1 - q0, (int64_t)a.max_q);
            it.k0 = (int)k0;
            it.off = (int)((k1 - k0) - (q1 - q0));   // (a cut by max_q moves no position)
            return it;
        }
        at += __shfl_sync(FULL, inc, 31);
    }
    return it;
}

// What the roles derive from an item
struct Range {
    int tB, last, kbeg, n;
    bool hasB;
    __device__ __forceinline__ Range(const Item &it, int nt, int window)
    {
        tB = it.tA + nt;
        hasB = tB < it.lq;
        last = min(it.tA + 2 * nt, it.lq) - 1;                   // last query token of the pair
        kbeg = window ? max(it.tA + it.off - window + 1, 0) : 0;
        const int kend = last + it.off + 1;
        n = kend > kbeg ? (kend - kbeg + kKeys - 1) / kKeys : 0;   // tiles of keys
    }
    // whether some row of the pair does not see all keys of tile j
    __device__ __forceinline__ bool masked(const Item &it, int window, int j) const
    {
        const int s = kbeg + j * kKeys;
        return s + kKeys - 1 > it.tA + it.off || (window && s < last + it.off - window + 1);
    }
};

constexpr int kItems = 2;   // items in hand: the one being worked on and the next

// bit 15 of each half set where its exponent is all ones (an infinity or NaN); other bits mean nothing
template <typename T>
__device__ __forceinline__ uint32_t exponent_full(uint32_t w)
{
    constexpr bool B = __is_same(T, __nv_bfloat16);
    return (w & (B ? 0x7f807f80u : 0x7c007c00u)) + (B ? 0x00800080u : 0x04000400u);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptK p)
{
    using L = PromptSmem<D>;
    constexpr int S = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Item s_items[kItems];
    __shared__ __align__(16) uint4 s_cancel;
    const maple_attn_prompt_args &a = p.a;
    // (a broadcast value is the same in a warp for the compiler too: the roles' code then counts as
    // convergent and may use uniform registers)
    const int warp = __shfl_sync(FULL, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (smem_addr(smem) & 1023u) {   // the swizzled tiles need 1024-byte alignment
        if (threadIdx.x == 0) set_flag(a.flags, MAPLE_DEVFLAG_TIMEOUT);
        return;
    }
    uint64_t *bars = (uint64_t *)(smem + L::kBars);
    const uint32_t b_full = smem_addr(bars), b_empty = b_full + 8 * S, b_q = b_empty + 8 * S, b_qfree = b_q + 8;
    const uint32_t b_s = b_qfree + 8, b_p = b_s + 16, b_pv = b_p + 16, b_item = b_pv + 16, b_ifree = b_item + 8 * kItems;
    const uint32_t b_cancel = b_ifree + 8 * kItems, b_drain = b_cancel + 8, b_next = b_drain + 8,
                   b_sfree = b_next + 8;
    uint32_t *tmem_holder = (uint32_t *)(bars + 2 * S + 2 + 2 + 2 + 2 + 2 * kItems + 4);
    volatile uint32_t *abort = tmem_holder + 1;
    uint32_t *odd_values = tmem_holder + 2;   // [2 items] something in V was not finite
    const uint64_t limit = kDefaultWaitNs;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(b_full + 8 * s, 1);
            mbar_init(b_empty + 8 * s, 1);
        }
        mbar_init(b_q, 1);
        mbar_init(b_qfree, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_p + 8 * i, 4);
            mbar_init(b_pv + 8 * i, 1);
        }
        for (int i = 0; i < kItems; i++) {
            mbar_init(b_item + 8 * i, 1);
            mbar_init(b_ifree + 8 * i, 10);   // loads, products, 8 softmax warps
            odd_values[i] = 0u;
        }
        mbar_init(b_cancel, 1);
        mbar_init(b_drain, 1);
        mbar_init(b_next, 1);
        mbar_init(b_sfree, 4);
        *abort = 0u;
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(smem_addr(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    constexpr uint32_t kP = 128, kO = 256;   // first columns of P_A and O_A (S: column 0)

    // the u-th item of this CTA, as the scheduling warp wrote it (false: a wait gave up)
    auto get_item = [&](int u, Item &it) -> bool {
        const int s = u % kItems;
        if (!mbar_wait(b_item + 8 * s, (u / kItems) & 1, abort, a.flags, limit)) return false;
        it = s_items[s];
        return true;
    };
    auto drop_item = [&](int u) { mbar_arrive(b_ifree + 8 * (u % kItems)); };   // by one lane of each reading warp

    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp == 10) {
        // ---------------- items: this block's own, then those of blocks that have not started
        int block = blockIdx.x, beyond = 0x7fffffff;   // blocks from `beyond` on have no item
        const uint64_t item_limit = 30 * limit;        // (these waits last as long as an item's loads)
        bool ok = true;
        for (int u = 0; ok; u++) {
            Item it;
            it.kvh = block >= 0 ? -2 : -1;
            if (block >= 0 && block < beyond) {
                it = find_item(a, p.nt, block);
                if (it.kvh == -2) beyond = block;
            }
            if (block == 0) {   // report offsets that are cut
                for (int b = lane; b < a.B; b += 32) {
                    const int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
                    if (q0 < 0 || q1 < q0 || q1 > a.Tq || q1 - q0 > a.max_q || k0 < 0 || k1 < k0 || k1 > a.Tk)
                        set_flag(a.flags, MAPLE_DEVFLAG_BAD_INDEX);
                }
            }
            const int s = u % kItems;
            ok = mbar_wait(b_ifree + 8 * s, ((u / kItems) & 1) ^ 1, abort, a.flags, item_limit);
            ok = __all_sync(FULL, ok);
            if (lane == 0 && ok) {
                s_items[s] = it;
                odd_values[s] = 0u;
                mbar_arrive(b_item + 8 * s);
            }
            if (block < 0 || !ok) break;
            // The next item is asked for when the last load of this one is issued: a whole item
            // ahead, the order of the items and not the CTAs' progress would decide who gets which.
            if (!__all_sync(FULL, mbar_wait(b_next, u & 1, abort, a.flags, item_limit))) break;
            if (lane == 0) {
                mbar_expect_tx(b_cancel, 16);
                try_cancel(smem_addr(&s_cancel), b_cancel);
            }
            // (waited for even after a failure: nothing may be in flight at the end)
            const uint64_t c0 = global_ns();
            bool got;
            while (!(got = mbar_test(b_cancel, u & 1)) && global_ns() - c0 < limit) {
            }
            block = __all_sync(FULL, got) ? cancelled_block(&s_cancel) : -1;
            __syncwarp();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the answer is read before it is overwritten
        }
      } else if (warp == 8) {
        // ---------------- loads
        // (one flat loop over the pairs of all items, here and in the products: the ring position is a
        // plain loop counter)
        if (lane == 0) {
            Item w;
            int u = -1, j = 0, n = -1, nq = 0, kbeg = 0;
            bool ok = true;
            for (uint32_t it = 0;; it++, j++) {   // pair it of the ring: K_j (j < n) and V_j-1 (j > 0), n + 1 pairs for an item
                bool done = false;
                while (j == n + 1) {
                    if (u >= 0) {
                        drop_item(u);
                        mbar_arrive(b_next);
                    }
                    u++;
                    if (!(ok = get_item(u, w)) || w.kvh == -1) {
                        done = true;
                        break;
                    }
                    const Range g(w, p.nt, a.window);
                    n = w.kvh >= 0 ? g.n : 0;
                    j = n > 0 ? 0 : n + 1;
                    kbeg = g.kbeg;
                    if (n > 0) {
                        if (!(ok = mbar_wait(b_qfree, (nq & 1) ^ 1, abort, a.flags, limit))) {
                            done = true;
                            break;
                        }
                        nq++;
                        mbar_expect_tx(b_q, (g.hasB ? 2 : 1) * L::kHalves * p.G * p.nt * 128);
                        for (int i = 0; i < (g.hasB ? 2 : 1); i++)
                            for (int h = 0; h < L::kHalves; h++)
                                tma_load_3d(smem_addr(smem + i * L::kTileBytes + h * 16384), &q_map, 64 * h, w.kvh * p.G,
                                            w.q0 + (i ? g.tB : w.tA), b_q);
                    }
                }
                if (done) break;
                const uint32_t s = it % S;
                if (!(ok = mbar_wait(b_empty + 8 * s, ((it / S) & 1) ^ 1, abort, a.flags, limit))) break;
                mbar_expect_tx(b_full + 8 * s, (j > 0 && j < n ? 2 : 1) * L::kTileBytes);
                const uint32_t dst = smem_addr(smem + L::kKv + s * 2 * L::kTileBytes);
                const int row = w.k0 + kbeg + j * kKeys;
                if (j < n)
                    for (int h = 0; h < L::kHalves; h++) tma_load_3d(dst + h * 16384, &k_map, 64 * h, w.kvh, row, b_full + 8 * s);
                if (j > 0)
                    for (int h = 0; h < L::kHalves; h++)
                        tma_load_3d(dst + L::kTileBytes + h * 16384, &v_map, 64 * h, w.kvh, row - kKeys, b_full + 8 * s);
            }
            if (*abort) {   // drain the copies in flight: whatever was asked of a barrier arrives or runs out of time
                for (int q = 0; q < S + 1; q++) {
                    const uint32_t bar = q < S ? b_full + 8 * q : b_q;
                    const uint64_t c0 = global_ns();
                    while (global_ns() - c0 < 20000000ull && !(mbar_test(bar, 0) && mbar_test(bar, 1))) {
                    }
                }
            }
        }
      } else if (warp == 9) {
        // ---------------- products
        // One elected lane of a warp whose index is a broadcast: the compiler then keeps the products'
        // operands in uniform registers.  (Without the broadcast they were moved there one by one,
        // 80 clocks a product; with all lanes running it, votes and reconvergence cost 100 clocks a wait.)
        const bool leader = elect_one();
        const bool bf = __is_same(T, __nv_bfloat16);
        const uint32_t id_s = idesc_f16(bf, kKeys, false), id_o = idesc_f16(bf, D, true);
        const uint32_t tm = __reduce_max_sync(FULL, tmem);   // (a warp reduction's result is in a uniform register)
        const uint64_t dq = desc_sw128(smem_addr(smem)), dk = desc_sw128(smem_addr(smem + L::kKv));
        const uint64_t dv = desc_mn_sw128(smem_addr(smem + L::kKv + L::kTileBytes));
        constexpr uint64_t kStep = L::kTileBytes / 16;   // a tile in descriptor units
        if (leader) {
        int u = -1, j = 0, n = -1, ni = 0;
        // pairs so far, tiles of A and of B (the phases of P), items with a Q, products into S
        uint32_t it = 0, phA = 0, phB = 0, nq = 0, nscore = 0;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return mbar_poll(bar, parity) || mbar_wait(bar, parity, abort, a.flags, limit);
        };
        // S = Q_i K^T of stage s, once the rows of the scores before have been taken out of S
        auto scores = [&](int i, uint32_t s) -> bool {
            if (nscore > 0 && !wait(b_sfree, (nscore - 1) & 1)) return false;
            nscore++;
            tc_fence_after();
            const uint64_t da = dq + i * kStep, db = dk + s * (2 * kStep);
#pragma unroll
            for (int k = 0; k < D / 16; k++)
                mma_ss(tm, da + (k / 4) * 1024 + 2 * (k % 4), db + (k / 4) * 1024 + 2 * (k % 4), id_s, k != 0);
            mma_commit(b_s + 8 * i);
            return true;
        };
        // O_i += P_i V of stage s
        auto values = [&](int i, uint32_t s, bool first) {
            const uint64_t db = dv + s * (2 * kStep);
#pragma unroll
            for (int k = 0; k < kKeys / 16; k++)
                mma_ts(tm + kO + D * i, tm + kP + 64 * i + 8 * k, db + 128 * k, id_o, k > 0 || !first);
            mma_commit(b_pv + 8 * i);
        };
        // Pair `it` of the ring holds K_j and V_j-1.  A step issues S = Q K_j and then O += P V_j-1
        // for A and for B, so that scores are computed while the rows of the tile before are in the
        // exponentials.  The stage is released and the next pair waited for behind the products of B,
        // while the tensor cores are still busy.
        bool ready = false;          // pair `it` has arrived
        for (;; it++, j++) {
            bool done = false;
            while (j == n + 1) {
                if (u >= 0) drop_item(u);
                u++;
                Item w;
                const bool got = get_item(u, w);
                if (!got || w.kvh == -1) {
                    done = true;
                    break;
                }
                const Range g(w, p.nt, a.window);
                n = w.kvh >= 0 ? g.n : 0;
                ni = g.hasB ? 2 : 1;
                j = n > 0 ? 0 : n + 1;
                if (n > 0) {
                    if (!wait(b_q, nq & 1)) {
                        done = true;
                        break;
                    }
                    nq++;
                }
            }
            if (done) break;
            const uint32_t s = it % S;
            if (!ready && !wait(b_full + 8 * s, (it / S) & 1)) break;
            bool ok = true;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                if (i == 0 || ni == 2) {
                    if (j < n) ok = ok && scores(i, s);
                    if (j > 0) {
                        ok = ok && wait(b_p + 8 * i, (i == 0 ? phA : phB) & 1);
                        if (ok) {
                            tc_fence_after();
                            values(i, s, j == 1);
                        }
                    }
                }
            }
            if (!ok) break;
            if (j > 0) {
                phA++;
                if (ni == 2) phB++;
            }
            mma_commit(b_empty + 8 * s);
            if (j + 1 == n) mma_commit(b_qfree);   // the last scores are issued
            ready = j < n && wait(b_full + 8 * ((it + 1) % S), ((it + 1) / S) & 1);
            if (j < n && !ready) break;
        }
        mma_commit(b_drain);   // every issued MMA has finished before tensor memory is released
        const uint64_t c0 = global_ns();
        while (!mbar_test(b_drain, 0) && global_ns() - c0 < limit) {
        }
        }
      }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      // ---------------- softmax and epilogue: one thread per row
      const int i = warp >> 2, r = threadIdx.x & 127;
      const int rt = r / p.G, h = r - rt * p.G;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes, tp = tmem + kP + 64 * i + lanes, to = tmem + kO + D * i + lanes;
      const bool neg = a.scale < 0.0f;
      const float scale2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);   // (0 as 10^-30: -inf stays -inf)
      uint32_t t0 = 0;            // ring position of the item's first pair
      uint32_t ns = 0;            // tiles of this half so far: the phase of S_i, P_i and O_i
      bool ok = true;
      for (int u = 0; ok; u++) {
        Item w;
        if (!(ok = __all_sync(FULL, get_item(u, w))) || w.kvh == -1) break;
        const Range g(w, p.nt, a.window);
        const int n = w.kvh >= 0 ? g.n : 0;
        if (w.kvh >= 0 && (i == 0 || g.hasB)) {
            const int tok = (i ? g.tB : w.tA) + rt;
            const bool valid = r < p.G * p.nt && tok < w.lq;
            const int pos = tok + w.off;                    // key position of the row's query
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; j++) {
                const bool edge = g.masked(w, a.window, j);
                ok = ok && mbar_wait(b_s + 8 * i, ns & 1, abort, a.flags, limit);
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                ns++;
                tc_fence_after();
                float s[kKeys];
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_ld32(ts + c, *reinterpret_cast<int(*)[32]>(&s[c]));
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_sfree);   // the next scores may be written
                if (neg) {
#pragma unroll
                    for (int c = 0; c < kKeys; c++) s[c] = -s[c];
                }
                if (edge) {   // the columns lo .. hi as one bit each
                    const int base = g.kbeg + j * kKeys, hi = pos - base, lo = a.window ? hi - a.window + 1 : 0;
#pragma unroll
                    for (int q = 0; q < kKeys; q += 32) {
                        const int h = hi - q, l0 = lo - q;
                        uint32_t keep = h >= 31 ? FULL : h < 0 ? 0u : (2u << h) - 1u;
                        keep &= l0 <= 0 ? FULL : l0 > 31 ? 0u : FULL << l0;
#pragma unroll
                        for (int c = 0; c < 32; c++)
                            if (!(keep & (1u << c))) s[q + c] = -INFINITY;
                    }
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; c++) mx[c] = max3(s[3 * c], s[3 * c + 1], s[3 * c + 2]);
#pragma unroll
                for (int c = 12; c < kKeys; c += 2) mx[(c / 2) & 3] = max3(mx[(c / 2) & 3], s[c], s[c + 1]);
                const float mt = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * scale2;
                // the products of the tile before have read P and updated O
                if (j > 0) ok = mbar_wait(b_pv + 8 * i, ns & 1, abort, a.flags, limit);
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                tc_fence_after();
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
                const float minus = m == -INFINITY ? 0.0f : kLift<T> - m;
                const uint64_t scale_2 = pair(scale2, scale2), minus_2 = pair(minus, minus);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < kKeys; c += 64) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        const uint64_t x = fma2(pair(s[c + e], s[c + e + 1]), scale_2, minus_2);
                        float p0, p1;
                        unpair(x, p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[(e / 2) & 1] = add2(sum[(e / 2) & 1], pair(p0, p1));
                        pk[e / 2] = Elem<T>::pack(p0, p1);
                    }
                    tmem_st32(tp + c / 2, pk);
                }
                tmem_wait_st();
                if (edge && i == 0) {
                    // V_j: what is not finite becomes 0 before the products read it (they wait for P of all
                    // four warps, so for all of the tile)
                    const uint32_t t = t0 + j + 1;       // (V_j comes with K_j+1)
                    if (!mbar_wait(b_full + 8 * (t % S), (t / S) & 1, abort, a.flags, limit)) ok = false;
                    uint4 *tile = (uint4 *)(smem + L::kKv + ((t % S) * 2 + 1) * L::kTileBytes);
                    constexpr int N16 = L::kTileBytes / 16 / 128;
                    uint32_t found = 0;
                    if (ok) {
#pragma unroll 2
                        for (int c = 0; c < N16; c++) {
                            const uint4 v = tile[threadIdx.x + 128 * c];
                            found |= exponent_full<T>(v.x) | exponent_full<T>(v.y) | exponent_full<T>(v.z) | exponent_full<T>(v.w);
                        }
                    }
                    if (found & 0x80008000u) {
                        for (int c = 0; c < N16; c++) {
                            const uint4 v = tile[threadIdx.x + 128 * c];
                            tile[threadIdx.x + 128 * c] = make_uint4(v.x & ~not_finite<T>(v.x), v.y & ~not_finite<T>(v.y),
                                                                     v.z & ~not_finite<T>(v.z), v.w & ~not_finite<T>(v.w));
                        }
                        atomicOr(odd_values + u % kItems, 1u);
                        fence_async_smem();
                    }
                    if (!__all_sync(FULL, ok)) break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p + 8 * i);
                float s0, s1;
                unpair(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
            }
            if (n > 0) {
                ok = ok && mbar_wait(b_pv + 8 * i, (ns - 1) & 1, abort, a.flags, limit);
            }
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            tc_fence_after();
            const bool none = l == 0.0f;    // the row sees no key
            const bool fix = n > 0 && *(volatile uint32_t *)(odd_values + u % kItems) != 0;
            const float inv = l > 0.0f || l != l ? __fdiv_rn(1.0f, l) : 0.0f;
            const int64_t row = (int64_t)(w.q0 + tok) * a.heads + w.kvh * p.G + h;
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
                        if (!g.masked(w, a.window, j)) continue;
                        const int s0 = max(g.kbeg + j * kKeys, from), s1 = min(g.kbeg + (j + 1) * kKeys, pos + 1);
                        for (int key = s0; key < s1; key++) {
                            const T *v = (const T *)a.v + (int64_t)(w.k0 + key) * a.v_stride + (int64_t)w.kvh * D + c;
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
                        for (int z = 0; z < 8; z++) y[z] = none ? 0.0f : o[e + z] * inv;
                        *reinterpret_cast<uint4 *>((T *)a.out + row * D + c + e) = pack8<T>(y);
                    }
                }
            }
            if (valid && a.lse) a.lse[row] = none ? -INFINITY : (m + (log2f(l) - kLift<T>)) * 0.6931471805599453f;
            tc_fence_before();   // O is read before the next item's first product writes it (ordered by P's barrier)
        }
        if (n > 0) t0 += n + 1;
        __syncwarp();
        if (lane == 0) drop_item(u);
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
        if (s % 8 || s <= 0 || s >= (1ll << 38)) return MAPLE_ERR_INVALID_ARG;
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
