// C ABI of the 8-bit paged attention: argument validation, workspace sizing and dispatch.
// The operations and their contracts are documented in include/attn.h.

#include <math.h>

#include "attn_internal.cuh"

namespace {

bool al16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

int check_cfg(const attn_config_t* c) {
    if (!c || c->num_q_heads <= 0 || c->num_kv_heads <= 0 || c->num_q_heads % c->num_kv_heads != 0)
        return GDN_ERR_INVALID_ARG;
    if (c->head_dim <= 0 || c->page_size <= 0 || isnan(c->scale) || isinf(c->scale) || isnan(c->logit_cap) ||
        isinf(c->logit_cap))
        return GDN_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return GDN_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return GDN_ERR_UNSUPPORTED;
    if (c->dtype != GDN_DTYPE_BF16 && c->dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
    if (c->num_kv_heads > 1024 || c->num_q_heads / c->num_kv_heads > 128) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

int elem_size(const attn_config_t* c) { return c->dtype == GDN_DTYPE_F32 ? 4 : 2; }

int check_cache(const attn_cache_t* c) {
    if (!c || !c->k || !c->v || !c->k_exp || !c->v_exp || c->num_pages <= 0) return GDN_ERR_INVALID_ARG;
    return al16(c->k) && al16(c->v) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

// a row stride in elements, resolved: 0 is contiguous; -1 for one that does not hold a row or is misaligned
int64_t resolve_stride(int64_t stride, int64_t row, int elem) {
    if (stride == 0) return row;
    if (stride < row || stride > ((int64_t)1 << 40) || stride * elem % 16 != 0) return -1;
    return stride;
}

// what either kernel needs for up to N requests and T rows (of any smaller batch too); a call that takes both takes them
// one after the other
size_t workspace_bytes(const attn_config_t* cfg, int64_t N, int64_t T) {
    const size_t split = gdn::attn::split_workspace_bytes(cfg->head_dim);
    const size_t tiles =
        gdn::attn::extend_workspace_bytes(cfg->head_dim, cfg->dtype, N, T * (cfg->num_q_heads / cfg->num_kv_heads));
    return split > tiles ? split : tiles;
}

struct Call {
    const attn_config_t* cfg;
    const attn_options_t* opts;
    const void* q;
    int64_t q_stride;
    const int32_t* cu;
    int per, N, T;
    const int32_t* kv_lens;
    const int32_t* table;
    int max_pages;
    const attn_cache_t* cache;
    const int32_t* parents;
    void* out;
    float* lse;
    void* ws;
    size_t ws_bytes, ws_need;
    gdn_stream_t stream;
};

// How a call's requests are shared out between the two: by their average, which for a ragged batch says nothing of any one
// of them.  From 2048 rows above one token per request (64 more passes over a cache, if one request has them), each goes to
// the kernel that its own rows ask for, at the price of three more launches: 256 requests of 2 rows, 16/2 heads, 107 us (all in
// tiles 190, as drafts to verify 91); 255 single rows and one request of 600 behind 8000 tokens, 32/8 heads, 384 us (788).
enum Kernels { kSplit, kTiles, kBoth };
Kernels kernels_for(const int32_t* cu, int64_t N, int64_t T, int64_t G, int split_rows) {
    if (T * G > split_rows * N) return kTiles;
    return cu && (T - N) * G >= 2048 ? kBoth : kSplit;
}

// Checks what the attending calls share and launches; an empty batch returns before its pointers are read.
int attend(const Call& c) {
    if (c.N < 0 || c.T < 0) return GDN_ERR_INVALID_ARG;
    if (!c.ws) return GDN_ERR_INVALID_ARG;
    if (c.N == 0 || c.T == 0) return GDN_OK;
    if (!al16(c.ws) || !c.q || !c.kv_lens || !c.table || !c.out || c.max_pages <= 0) return GDN_ERR_INVALID_ARG;
    int rc = check_cache(c.cache);
    if (rc != GDN_OK) return rc;
    const void* ptrs[] = {c.q, c.cu, c.kv_lens, c.table, c.parents, c.out, c.lse,
                          c.opts ? c.opts->slopes : nullptr, c.opts ? c.opts->prefix_lens : nullptr};
    for (const void* q : ptrs)
        if (q && !al16(q)) return GDN_ERR_INVALID_ARG;
    const int D = c.cfg->head_dim;
    const int64_t qs = resolve_stride(c.q_stride, (int64_t)c.cfg->num_q_heads * D, elem_size(c.cfg));
    if (qs < 0) return GDN_ERR_INVALID_ARG;
    if ((int64_t)c.max_pages * c.cfg->page_size > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    const int G = c.cfg->num_q_heads / c.cfg->num_kv_heads;
    if ((int64_t)c.T * G >= (1 << 25) || c.N > (1 << 28)) return GDN_ERR_UNSUPPORTED;
    if (c.ws_bytes < c.ws_need) return GDN_ERR_WORKSPACE;

    gdn::attn::Args a{};
    a.HQ = c.cfg->num_q_heads;
    a.HKV = c.cfg->num_kv_heads;
    a.G = G;
    a.g_inv = G == 1 ? 0u : (uint32_t)(((1ull << 32) + G - 1) / G);
    a.ps_shift = log2_of(c.cfg->page_size);
    a.window = c.cfg->window;
    a.scale2 = (c.cfg->scale > 0.0f ? c.cfg->scale : 1.0f / sqrtf((float)D)) * gdn::attn::kLog2e;
    // (a cap outside the limits makes every score zero, or changes none; within them nothing overflows in the kernels)
    a.cap2 = c.cfg->logit_cap > 0.0f ? fminf(fmaxf(c.cfg->logit_cap * gdn::attn::kLog2e, 0x1p-100f), 0x1p120f) : 0.0f;
    a.q = c.q;
    a.q_stride = qs;
    a.cu = c.cu;
    a.per = c.per;
    a.N = c.N;
    a.T = c.T;
    a.kv_lens = c.kv_lens;
    a.table = c.table;
    a.max_pages = c.max_pages;
    a.k = static_cast<const uint8_t*>(c.cache->k);
    a.v = static_cast<const uint8_t*>(c.cache->v);
    a.k_exp = c.cache->k_exp;
    a.v_exp = c.cache->v_exp;
    a.num_pages = c.cache->num_pages;
    a.slopes = c.opts ? c.opts->slopes : nullptr;
    a.prefix = c.opts ? c.opts->prefix_lens : nullptr;
    a.parents = c.parents;
    a.out = c.out;
    a.lse = c.lse;
    a.hdr = static_cast<int32_t*>(c.ws);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(c.stream);
    gdn::mark_launch(s, 0);
    const int split_rows = gdn::attn::split_rows(D, c.cfg->dtype == GDN_DTYPE_F32);
    const Kernels kernels = kernels_for(c.cu, c.N, c.T, G, split_rows);
    a.rows_upto = a.rows_above = kernels == kBoth ? split_rows : kernels == kTiles ? 0 : INT32_MAX;
    cudaError_t e = cudaSuccess;
    if (kernels != kTiles) e = gdn::attn::launch_split(a, D, c.cfg->dtype, s);
    if (kernels != kSplit && e == cudaSuccess) e = gdn::attn::launch_extend_tc(a, D, c.cfg->dtype, s);
    gdn::mark_launch(s, 1);
    return e == cudaSuccess ? GDN_OK : gdn::record_cuda_failure(e);
}

int verify(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride,
           const int32_t* parents, int32_t B, int32_t D, const int32_t* kv_lens, const int32_t* block_table,
           int32_t max_pages, const attn_cache_t* cache, void* out, float* lse, void* ws, size_t ws_bytes,
           gdn_stream_t stream) {
    const int rc = check_cfg(cfg);
    if (rc != GDN_OK) return rc;
    if (D < 1 || D > gdn::kMaxVerifyDraft || B < 0) return GDN_ERR_INVALID_ARG;
    if ((int64_t)B * D > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    return attend(Call{cfg, opts, q, q_stride, nullptr, D, B, B * D, kv_lens, block_table, max_pages, cache, parents, out,
                       lse, ws, ws_bytes, attn_verify_workspace_size(cfg, B, D), stream});
}

}  // namespace

extern "C" {

size_t attn_append_workspace_size(const attn_config_t* cfg, int32_t max_N, int32_t max_T) {
    if (check_cfg(cfg) != GDN_OK || max_N < 0 || max_T < 0) return 0;
    return gdn::kHeaderBytes;
}

int attn_append(const attn_config_t* cfg, const attn_cache_t* cache, const void* k_new, const void* v_new,
                int64_t k_stride, int64_t v_stride, const int32_t* cu_seqlens, int32_t N, int32_t T,
                const int32_t* start_lens, const int32_t* block_table, int32_t max_pages, void* workspace,
                size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_cfg(cfg);
    if (rc != GDN_OK) return rc;
    if (N < 0 || T < 0 || !workspace) return GDN_ERR_INVALID_ARG;
    if (!cu_seqlens && N > 0 && T % N != 0) return GDN_ERR_INVALID_ARG;
    if (N == 0 || T == 0) return GDN_OK;
    if (!al16(workspace) || !k_new || !v_new || !start_lens || !block_table || max_pages <= 0)
        return GDN_ERR_INVALID_ARG;
    rc = check_cache(cache);
    if (rc != GDN_OK) return rc;
    const void* ptrs[] = {k_new, v_new, cu_seqlens, start_lens, block_table};
    for (const void* q : ptrs)
        if (q && !al16(q)) return GDN_ERR_INVALID_ARG;
    const int64_t row = (int64_t)cfg->num_kv_heads * cfg->head_dim;
    const int64_t ks = resolve_stride(k_stride, row, elem_size(cfg)), vs = resolve_stride(v_stride, row, elem_size(cfg));
    if (ks < 0 || vs < 0) return GDN_ERR_INVALID_ARG;
    if ((int64_t)max_pages * cfg->page_size > (1 << 30) || N > (1 << 28) || T > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    if (workspace_bytes < attn_append_workspace_size(cfg, N, T)) return GDN_ERR_WORKSPACE;

    gdn::attn::AppendArgs a{};
    a.HKV = cfg->num_kv_heads;
    a.ps_shift = log2_of(cfg->page_size);
    a.x[0] = k_new;
    a.x[1] = v_new;
    a.stride[0] = ks;
    a.stride[1] = vs;
    a.codes[0] = static_cast<uint8_t*>(cache->k);
    a.codes[1] = static_cast<uint8_t*>(cache->v);
    a.exps[0] = cache->k_exp;
    a.exps[1] = cache->v_exp;
    a.cu = cu_seqlens;
    a.per = T / N;
    a.N = N;
    a.T = T;
    a.start = start_lens;
    a.table = block_table;
    a.max_pages = max_pages;
    a.num_pages = cache->num_pages;
    a.hdr = static_cast<int32_t*>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    gdn::mark_launch(s, 0);
    const cudaError_t e = gdn::attn::launch_append(a, cfg->head_dim, cfg->dtype, s);
    gdn::mark_launch(s, 1);
    return e == cudaSuccess ? GDN_OK : gdn::record_cuda_failure(e);
}

size_t attn_extend_workspace_size(const attn_config_t* cfg, int32_t max_N, int32_t max_T) {
    if (check_cfg(cfg) != GDN_OK || max_N < 0 || max_T < 0) return 0;
    return workspace_bytes(cfg, max_N, max_T);
}

int attn_extend(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride,
                const int32_t* cu_seqlens, int32_t N, int32_t T, const int32_t* kv_lens, const int32_t* block_table,
                int32_t max_pages, const attn_cache_t* cache, void* out, float* lse, void* workspace,
                size_t workspace_bytes, gdn_stream_t stream) {
    const int rc = check_cfg(cfg);
    if (rc != GDN_OK) return rc;
    if (N > 0 && T > 0 && !cu_seqlens) return GDN_ERR_INVALID_ARG;
    return attend(Call{cfg, opts, q, q_stride, cu_seqlens, 0, N, T, kv_lens, block_table, max_pages, cache, nullptr, out,
                       lse, workspace, workspace_bytes, attn_extend_workspace_size(cfg, N, T), stream});
}

size_t attn_decode_workspace_size(const attn_config_t* cfg, int32_t max_B) {
    if (check_cfg(cfg) != GDN_OK || max_B < 0) return 0;
    return workspace_bytes(cfg, max_B, max_B);
}

int attn_decode(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride, int32_t B,
                const int32_t* kv_lens, const int32_t* block_table, int32_t max_pages, const attn_cache_t* cache,
                void* out, float* lse, void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
    const int rc = check_cfg(cfg);
    if (rc != GDN_OK) return rc;
    return attend(Call{cfg, opts, q, q_stride, nullptr, 1, B, B, kv_lens, block_table, max_pages, cache, nullptr, out,
                       lse, workspace, workspace_bytes, attn_decode_workspace_size(cfg, B), stream});
}

size_t attn_verify_workspace_size(const attn_config_t* cfg, int32_t max_B, int32_t D) {
    if (check_cfg(cfg) != GDN_OK || max_B < 0 || D < 1 || D > gdn::kMaxVerifyDraft) return 0;
    return workspace_bytes(cfg, max_B, (int64_t)max_B * D);
}

int attn_verify(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride, int32_t B,
                int32_t D, const int32_t* kv_lens, const int32_t* block_table, int32_t max_pages,
                const attn_cache_t* cache, void* out, float* lse, void* workspace, size_t workspace_bytes,
                gdn_stream_t stream) {
    return verify(cfg, opts, q, q_stride, nullptr, B, D, kv_lens, block_table, max_pages, cache, out, lse, workspace,
                  workspace_bytes, stream);
}

int attn_verify_tree(const attn_config_t* cfg, const attn_options_t* opts, const void* q, int64_t q_stride,
                     const int32_t* parents, int32_t B, int32_t D, const int32_t* kv_lens, const int32_t* block_table,
                     int32_t max_pages, const attn_cache_t* cache, void* out, float* lse, void* workspace,
                     size_t workspace_bytes, gdn_stream_t stream) {
    if (B > 0 && !parents) return GDN_ERR_INVALID_ARG;
    return verify(cfg, opts, q, q_stride, parents, B, D, kv_lens, block_table, max_pages, cache, out, lse, workspace,
                  workspace_bytes, stream);
}

}  // extern "C"
