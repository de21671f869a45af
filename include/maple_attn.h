/*
 * maple_attn.h -- C ABI of the attention half of a decoder layer on B200
 * (sm_100a): the int8 projection, the per-head norm with the rotation by
 * position, a paged cache of 4-bit keys and values, attention over whole
 * prompts and attention of one new token per sequence over the cache.
 *
 * The model these stand next to has windowed layers (512 tokens) and global
 * ones in a 3:1 ratio over long contexts ("linlog.top/article/1232", section
 * 架构设计, model table); the pages give no interface, head layout or cache
 * format, so those are this library's own.
 *
 * Conventions (those of maple_moe.h, without a handle):
 *  - All tensor pointers are DEVICE pointers on the current CUDA device,
 *    16-byte aligned, owned by the caller.  Nothing is kept between calls.
 *  - Every call is asynchronous on the given stream, allocates nothing and
 *    never synchronises; all of them may be captured into a CUDA graph.
 *  - Scratch memory is the caller's too (`workspace`): two calls whose work
 *    may overlap on the GPU need two workspaces.  Its contents need no
 *    initialisation and mean nothing after the call.
 *  - Return value: MAPLE_OK or a negative MAPLE_ERR_* code of maple_moe.h.
 *    Values that only the device can see are checked by the kernels, which
 *    never read or write out of range: a bad index raises MAPLE_FLAG_BAD_INDEX
 *    and an expired bounded wait MAPLE_FLAG_TIMEOUT in *flags (a DEVICE word,
 *    may be NULL; bits are only ever set, the caller clears it).  The outputs
 *    of a call that raised MAPLE_FLAG_TIMEOUT are not valid.
 *
 * Head layout: `heads` query heads in `kv_heads` groups of heads/kv_heads;
 * query head h reads key/value head h / (heads/kv_heads).  head_dim is 64 or
 * 128.  A token's heads are contiguous; the step from token to token is a
 * stride in elements (a multiple of 8; positive in maple_attn_prompt), so views
 * of one fused projection are taken as they are.
 */
#ifndef MAPLE_ATTN_H
#define MAPLE_ATTN_H

#include "maple_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
enum { MAPLE_BF16 = 0, MAPLE_FP16 = 1, MAPLE_FP32 = 2 };

/*
 * The cache of 4-bit keys and values: uint8 [num_pages][kv_heads][page bytes],
 * page_size tokens (16, 32 or 64) to a page, page bytes = page_size * head_dim
 * * 5/4.  Token slot s is row p = s % page_size of page s / page_size.
 *
 * Values: for each token, head and 32 channels, minimum = fp16(min x) and
 * scale = fp16((max x - minimum)/15); code = rint((x - minimum)/scale) clamped
 * to 0..15 (0 where scale <= 0); the cache stands for minimum + scale * code.
 * x is clamped to +-60000 first; 32 channels with a NaN among them are all NaN.
 *
 * A page of one head, with d = head_dim, n = page_size, "word w" = the 8 codes
 * of channels 8w..8w+7 (channel 8w+i in bits 4i..4i+3), g = w/4, t = w%4:
 *   [n][d/2]         key codes: word w of row p at p*d/2 + (t*(d/32) + g)*4
 *   [n/16][8*d]      value codes in blocks of 16 rows (below)
 *   [n][d/32][2]     fp16 (scale, minimum) of the keys
 *   [d/32][n]        fp16 scales of the values
 *   [d/32][n]        fp16 minima of the values
 * Value codes of row r = p%16 of a block, with u = (r%8)/2, z = r%2 + 2*(r/8):
 *   d = 128: word w at (z/2)*512 + ((w/2)*4 + u)*16 + (z%2)*8 + (w%2)*4
 *   d =  64: word w at (w*4 + u)*16 + z*4
 * (the order in which the lanes of a warp-level matrix instruction want them).
 */

/* Bytes of one page of one head, or MAPLE_ERR_UNSUPPORTED_SHAPE. */
int64_t maple_attn_page_bytes(int32_t head_dim, int32_t page_size);

/*
 * y[t][n] = f32(sum_k w[n][k] q[t][k]) * (alpha[n] * s[t]) (+ bias[n])
 * (+ resid[t][n]), with q, s the int8 absmax codes of row t of x (scale
 * amax/127, a zero row gives 0): the quantiser and the order of the roundings
 * are those of the expert matrices, and the sum is exact.
 * normalise != 0: x is the fp32 residual stream and the row that is quantised
 * is bf16(RMSNorm(x)) (norm weights 1, eps 1e-6, the layer stack's rule; K must
 * be a multiple of 256 then).
 * A row of x that holds a NaN or an infinity gives a row of NaN, with normalise
 * also one whose sum of squares is beyond fp32 (values of 10^18 and more).
 * resid may be y; y overlaps nothing else that the call reads.
 * Limits: K a multiple of 16, 16 <= K <= 32768; 1 <= N; T*N and N*K < 2^40.
 * T == 0 is a no-op.
 */
typedef struct {
    const void *x;          /* [T] rows of K: bf16, or fp32 with normalise */
    const int8_t *w;        /* [N][K] */
    const float *alpha;     /* [N] */
    const float *bias;      /* [N] or NULL */
    const float *resid;     /* [T][N] fp32 or NULL */
    void *y;                /* [T][N] of y_dtype */
    void *workspace;        /* maple_attn_linear_workspace bytes; NULL where that is 0 */
    int64_t workspace_bytes;
    uint32_t *flags;
    int64_t x_stride;       /* elements from row to row of x (a multiple of 8) */
    int64_t T, K, N;
    int32_t y_dtype;        /* MAPLE_BF16 or MAPLE_FP32 */
    int32_t normalise;
} maple_attn_linear_args;

/* Bytes of workspace that a call needs (0: none), or a negative MAPLE_ERR_* code. */
int64_t maple_attn_linear_workspace(int64_t T, int64_t K, int64_t N, int32_t normalise);
int maple_attn_linear(const maple_attn_linear_args *args, maple_stream_t stream);

/*
 * Per head of q and of k: x / sqrt(mean(x^2) + eps) * weight, then the first
 * rotary_dim channels rotated in pairs by the angle position * inv_freq[i]
 * (pairs (i, i + rotary_dim/2), or (2i, 2i+1) with interleaved), rounded once.
 * With `pages` the rotated keys (as rounded to dtype) and the values are also
 * written to the cache at `slots` (< 0: that token is not stored; a slot beyond
 * the cache is not stored and raises MAPLE_FLAG_BAD_INDEX).  The slots of one
 * call must be distinct: two tokens on one slot leave a mix of their codes.
 * rotary_dim is a multiple of 16 up to head_dim (0: no rotation).
 */
typedef struct {
    const void *q, *k, *v;          /* [T][heads][d], [T][kv_heads][d]; v only with pages */
    void *q_out, *k_out;            /* [T][heads][d], [T][kv_heads][d], contiguous; k_out may be NULL with pages */
    const float *q_weight, *k_weight;   /* [d] or NULL (1) */
    const int64_t *positions;       /* [T] */
    const double *inv_freq;         /* [rotary_dim/2], radians per position */
    uint8_t *pages;                 /* the cache or NULL */
    const int64_t *slots;           /* [T] */
    uint32_t *flags;
    int64_t q_stride, k_stride, v_stride;   /* elements from token to token */
    int64_t T, num_pages;
    int32_t heads, kv_heads, head_dim, rotary_dim, page_size, dtype, interleaved;
    float eps;
} maple_attn_rope_args;

int maple_attn_qk_norm_rope(const maple_attn_rope_args *args, maple_stream_t stream);

/*
 * The values that the cache holds at `slots`, rounded once to dtype: k, v
 * [n][kv_heads][d] contiguous.  A negative slot reads as zeros, one beyond the
 * cache too (and raises MAPLE_FLAG_BAD_INDEX).
 */
typedef struct {
    const uint8_t *pages;
    const int64_t *slots;           /* [n] */
    void *k, *v;
    uint32_t *flags;
    int64_t n, num_pages;
    int32_t kv_heads, head_dim, page_size, dtype;
} maple_attn_read_args;

int maple_attn_kv_read(const maple_attn_read_args *args, maple_stream_t stream);

/*
 * Causal attention over packed sequences.  Sequence b has the query rows
 * cu_q[b] .. cu_q[b+1]-1 and the key rows cu_k[b] .. cu_k[b+1]-1; its queries
 * are its last positions: query i (of lq) stands at key position i + lk - lq
 * and sees the keys j with position - window < j <= position (window == 0: all
 * j <= position).  A query that sees no key gives a row of zeros and lse -inf.
 * out[t][h] = sum_j softmax_j(scale * q.k_j) v_j; lse (may be NULL) fp32
 * [Tq][heads] = log sum_j exp(scale * q.k_j).  Rows of out and lse that belong
 * to no sequence are left as they were; out and lse overlap nothing that the
 * call reads.  What stands in masked keys and values
 * (infinities, NaN) does not reach the output.
 * Limits: at most 64 query heads per key/value head and 1024 in all, 65535
 * sequences, 2^30 rows of queries and of keys.
 * max_q bounds every lq from above (a sequence with more query rows raises
 * MAPLE_FLAG_BAD_INDEX and loses the rows beyond max_q); offsets that fall or
 * reach beyond Tq or Tk are cut to them and raise MAPLE_FLAG_BAD_INDEX.
 */
typedef struct {
    const void *q, *k, *v;          /* [Tq][heads][d], [Tk][kv_heads][d] */
    void *out;                      /* [Tq][heads][d] contiguous */
    float *lse;
    const int32_t *cu_q, *cu_k;     /* [B+1] */
    uint32_t *flags;
    int64_t q_stride, k_stride, v_stride;
    int64_t Tq, Tk;
    int32_t B, max_q, heads, kv_heads, head_dim, window, dtype;
    float scale;
} maple_attn_prompt_args;

int maple_attn_prompt(const maple_attn_prompt_args *args, maple_stream_t stream);

/*
 * One new token per sequence: q [B][heads][d] at position lens[b]-1, over the
 * lens[b] cached tokens of sequence b (its own key and value included, so they
 * are appended first); position j sits in page block_table[b][j/page_size].
 * window as above.  lens[b] <= 0 gives a row of zeros; lens[b] is cut to
 * max_pages*page_size (MAPLE_FLAG_BAD_INDEX).  A page number outside the cache
 * is skipped as if its positions were masked (MAPLE_FLAG_BAD_INDEX).
 * Limits: 1024 query heads, 65535 sequences, max_pages * page_size <= 2^30.
 */
typedef struct {
    const void *q;                  /* [B][heads][d] */
    void *out;                      /* [B][heads][d] contiguous */
    const uint8_t *pages;
    const int32_t *block_table;     /* [B][max_pages] (table_stride from row to row) */
    const int32_t *lens;            /* [B] */
    void *workspace;                /* maple_attn_cached_workspace bytes; NULL where that is 0 */
    int64_t workspace_bytes;
    uint32_t *flags;
    int64_t q_stride, table_stride, num_pages;
    int32_t B, max_pages, heads, kv_heads, head_dim, page_size, window, dtype;
    float scale;
} maple_attn_cached_args;

int64_t maple_attn_cached_workspace(int32_t B, int32_t max_pages, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                    int32_t page_size, int32_t window);
int maple_attn_cached(const maple_attn_cached_args *args, maple_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAPLE_ATTN_H */
