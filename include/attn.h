/*
 * attn.h -- C ABI of the full-attention layers of a hybrid model in libgdn.so (sm_100a): a paged
 * key/value cache held in 8 bits, and the softmax attention that reads it.
 *
 * These are the layers that page "pymllm.layers.attention.hybrid_backend" sends to its full-attention
 * backend (forward_extend / forward_decode) beside the linear layers of gdn.h, with the conventions of
 * page "pymllm.layers.attention.radix_attention" (RadixAttention: grouped heads, scaling, logit_cap,
 * sliding window).  They have the forward modes of gdn.h:
 *
 *   attn_append       quantise new key and value rows into the cache (before each of the others)
 *   attn_extend       EXTEND: ragged packed rows over cached prefixes
 *   attn_decode       DECODE: one row per request
 *   attn_verify       TARGET_VERIFY: D draft rows per request (attn_verify_tree: a tree of drafts)
 *
 * The cache.  Pools of pages of `page_size` tokens, shared by all requests:
 *     k, v          [num_pages, HKV, page_size, head_dim]  e4m3 codes (1 byte each)
 *     k_exp, v_exp  [num_pages, HKV]                       int8 exponents in ATTN_EXP_MIN .. ATTN_EXP_MAX
 * A cached value is code * 2^exp: one power-of-two scale per page and head, keys and values apart, so
 * that only the rounding to e4m3 itself loses bits.  Token t of request n is row t % page_size of page
 * block_table[n][t / page_size] (int32 [N, max_pages], row-major).  Codes of live rows are finite:
 * attn_append writes nothing else.  Rows behind a request's length and pages that no row of a call sees
 * are never used and may hold anything, NaN codes included; their block_table entries may hold anything
 * too (-1, say).
 *
 * What a call computes.  Row i of request n is the query at position p_i of that request; query head h
 * reads key/value head h / (HQ/HKV):
 *     s_ij = scale * q_i . k_j;   s_ij = cap * tanh(s_ij / cap)  (logit_cap > 0)
 *     s_ij = s_ij - slopes[h] * |p_i - p_j|                      (slopes given)
 *     row i sees token j when  (p_j <= p_i  and  (window <= 0 or p_i - p_j < window))
 *                              or  p_j < prefix_lens[n]          (prefix_lens given: a prefix mask)
 *     out_i = sum_j softmax_j(s_ij) v_j;    lse_i = log sum_j exp(s_ij)
 * over the tokens it sees, among the kv_lens[n] tokens cached for request n (this call's own rows
 * included, appended before the call).  A row that sees nothing gets out = 0 and lse = -inf.  No row
 * sees another request's tokens: packed documents are requests of their own.
 *
 * Arithmetic.  Queries are scaled per row by a power of two and rounded to fp16 (exact for bf16 queries
 * down to 2^-28 of the row's largest; for fp32 queries a second fp16 takes the remainder), codes are
 * exact in fp16, products accumulate in fp32 (on the tensor core, whose additions truncate, over at most 512 tokens for
 * fp32, 32768 for bf16; those sums are added up with rounding), the softmax statistics are fp32, weights are rounded to
 * fp16 (for fp32 a second fp16 takes their remainder), the output is rounded once to the dtype.  A token's
 * weight times its value page's scale keeps all those bits down to 2^-14 (fp32: 2^-26) of the largest such
 * product of its row; below that it is off by at most 2^-25 (2^-37) of that product.
 * A capped score is off by at most 2^-20 of the score itself (bf16 with caps up to 256: 2^-20 of the cap).
 *
 * Conventions (as in gdn.h): every pointer is device memory owned by the caller and 16-byte aligned
 * (k_exp and v_exp: any alignment); calls are asynchronous and ordered on `stream`, allocate nothing and
 * may be captured into a CUDA graph; the workspace starts with the sticky device error word read by
 * gdn_get_device_error() and cleared by gdn_reset_device_error().  Its other contents need not outlive a
 * call; calls that may overlap on the GPU need workspaces of their own.  Argument errors return a
 * GDN_ERR_* code with nothing launched.
 *   - A request with kv_lens[n] < 0 (attn_append: start_lens[n] < 0) is padding: its output rows are
 *     zeros (lse -inf), nothing is appended for it.  kv_lens[n] == 0: the same.
 *   - kv_lens[n] (attn_append: start + rows) above max_pages * page_size, or below the request's row
 *     count, raises GDN_DEVERR_KV_LEN and the request is treated as padding.  (Of a request without rows no length is
 *     looked at: it may be a finished one's.)
 *   - A needed block_table entry outside 0 .. num_pages-1 raises GDN_DEVERR_PAGE_RANGE; its tokens are
 *     not read (attn_append: not written), and that request's outputs are invalid.
 *   - cu_seqlens must start at 0, not decrease, and end at or before T; otherwise GDN_DEVERR_SEQLENS is
 *     raised and the call does nothing.  Rows from cu_seqlens[N] on (a padded batch) are left as they
 *     were, in `out`, `lse` and the cache.
 * Rows of q, k_new and v_new may be further apart than their heads need (slices of a fused projection):
 * the *_stride arguments give the distance between rows in elements, 0 for contiguous rows; a row's
 * byte distance must be a multiple of 16.  out is contiguous [T, HQ, head_dim].  T * (HQ / HKV) must be below
 * 2^25 (attn_append: T at most 2^30), max_pages * page_size at most 2^30 and N at most 2^28 (GDN_ERR_UNSUPPORTED).
 * Waits inside the kernels give up after two seconds (GDN_DEVERR_TIMEOUT; results are invalid): rows that read more than
 * some 5 * 10^7 tokens of one request in one call can take a block that long.
 */
#ifndef ATTN_H
#define ATTN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* device error bits of these calls, in the same word as gdn.h's */
#define GDN_DEVERR_KV_LEN 0x80      /* a length outside its block table or below its row count; padded */
#define GDN_DEVERR_PAGE_RANGE 0x100 /* a needed block_table entry outside 0 .. num_pages-1 */
#define GDN_DEVERR_NONFINITE 0x200  /* attn_append met an inf or NaN (stored as the largest code, as 0) */

/* exponents of a block: amax <= 448 * 2^exp; smaller blocks use ATTN_EXP_MIN, larger values saturate */
#define ATTN_EXP_MIN (-32)
#define ATTN_EXP_MAX 60

typedef struct {
    int32_t num_q_heads;  /* HQ */
    int32_t num_kv_heads; /* HKV, divides HQ; HQ / HKV <= 128 */
    int32_t head_dim;     /* 64 or 128, keys and values alike */
    int32_t page_size;    /* tokens per page: 16, 32, 64 or 128 */
    int32_t dtype;        /* GDN_DTYPE_BF16 or GDN_DTYPE_F32: q, out, k_new, v_new */
    int32_t window;       /* tokens a row sees, itself included; <= 0: all before it */
    float scale;          /* <= 0: 1/sqrt(head_dim) */
    float logit_cap;      /* <= 0: none */
} attn_config_t;

typedef struct {
    void* k;            /* [num_pages, HKV, page_size, head_dim] e4m3 */
    void* v;            /* likewise */
    int8_t* k_exp;      /* [num_pages, HKV] */
    int8_t* v_exp;      /* [num_pages, HKV] */
    int32_t num_pages;
} attn_cache_t;

/* per-call options; a NULL pointer to it, or a NULL field, leaves the option out */
typedef struct {
    const float* slopes;        /* [HQ] distance bias per query head */
    const int32_t* prefix_lens; /* [N] tokens visible to every row of the request */
} attn_options_t;

/* Workspace bytes of attn_append (the error header only); 0 for an invalid configuration. */
GDN_API size_t attn_append_workspace_size(const attn_config_t* cfg, int32_t max_N, int32_t max_T);

/*
 * Quantises the rows k_new, v_new [T, HKV, head_dim] into the cache: request n's rows
 * cu_seqlens[n] .. cu_seqlens[n+1]-1 become its tokens start_lens[n], start_lens[n] + 1, ...
 * cu_seqlens NULL: T / N rows for each request (T a multiple of N; T == N is a decode step).
 * A page whose first token is written takes the smallest exponent e with amax <= 448 * 2^e over its new
 * rows.  A page that already holds tokens before the first new one keeps or raises its exponent, and when
 * it is raised those tokens' codes are rounded again to the nearest even code of the same value.  Tokens
 * from start + rows on are dropped (their rows keep stale codes), so a rejected draft is replaced by
 * appending at its position.  What it did to the page it began in stays, if tokens before it are there: an exponent
 * that it raised, and those tokens' values, which that exponent's smallest step, 2^(exp - 9), moved by up to half of
 * it.  (To be free of that, begin drafts on a page of their own, or append the page again from its first token.)
 * Two requests that write the same page race; full pages may be shared.
 */
GDN_API int attn_append(const attn_config_t* cfg, const attn_cache_t* cache, const void* k_new, const void* v_new,
                        int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens, int32_t N, int32_t T,
                        const int32_t* start_lens, const int32_t* block_table, int32_t max_pages, void* workspace,
                        size_t workspace_bytes, gdn_stream_t stream);

/* Workspace bytes of attn_extend over at most max_N requests and max_T packed rows. */
GDN_API size_t attn_extend_workspace_size(const attn_config_t* cfg, int32_t max_N, int32_t max_T);

/*
 * EXTEND: request n owns the packed rows cu_seqlens[n] .. cu_seqlens[n+1]-1 of q [T, HQ, head_dim], which
 * are its last tokens: with L rows, row r is at position kv_lens[n] - L + r.  out [T, HQ, head_dim];
 * lse [T, HQ] fp32 or NULL.
 */
GDN_API int attn_extend(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride,
                        const int32_t* cu_seqlens, int32_t N, int32_t T, const int32_t* kv_lens,
                        const int32_t* block_table, int32_t max_pages, const attn_cache_t* cache, void* out,
                        float* lse, void* workspace, size_t workspace_bytes, gdn_stream_t stream);

/* Workspace bytes of attn_decode over at most max_B requests. */
GDN_API size_t attn_decode_workspace_size(const attn_config_t* cfg, int32_t max_B);

/* DECODE: one row per request, its last token (position kv_lens[n] - 1).  q, out [B, HQ, head_dim]. */
GDN_API int attn_decode(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride,
                        int32_t B, const int32_t* kv_lens, const int32_t* block_table, int32_t max_pages,
                        const attn_cache_t* cache, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        gdn_stream_t stream);

/* Workspace bytes of attn_verify and attn_verify_tree over at most max_B requests of D drafts. */
GDN_API size_t attn_verify_workspace_size(const attn_config_t* cfg, int32_t max_B, int32_t D);

/*
 * TARGET_VERIFY: request n has D draft rows (rows n*D .. n*D+D-1 of q [B*D, HQ, head_dim]), its last D
 * tokens in order; kv_lens[n] counts them.  1 <= D <= 16.  The same result as attn_extend of D rows each.
 */
GDN_API int attn_verify(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride,
                        int32_t B, int32_t D, const int32_t* kv_lens, const int32_t* block_table, int32_t max_pages,
                        const attn_cache_t* cache, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        gdn_stream_t stream);

/*
 * TARGET_VERIFY over a draft tree, as gdn_verify_tree: draft t of request n continues parents[n*D + t]
 * (-1: the token before the drafts; otherwise an earlier draft).  With b = kv_lens[n] - D, draft t sees
 * the tokens before b, its ancestors and itself, and stands at position b + depth(t), depth being its
 * number of ancestors among the drafts; window and slopes go by these positions, prefix_lens by the order
 * in the cache.  A parent outside -1 .. t-1 raises GDN_DEVERR_TREE and the request is treated as padding.
 * To keep an accepted path, append its rows at position b again, in order.
 */
GDN_API int attn_verify_tree(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride,
                             const int32_t* parents, int32_t B, int32_t D, const int32_t* kv_lens,
                             const int32_t* block_table, int32_t max_pages, const attn_cache_t* cache, void* out,
                             float* lse, void* workspace, size_t workspace_bytes, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H */
