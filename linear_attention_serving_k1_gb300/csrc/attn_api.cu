// attn_api.cu -- C entry points of the attention layers: argument validation,
// workspace layout and kernel dispatch, in the manner of gdn_api.cu.
#include <math.h>

#include "attn.cuh"

namespace {

using kda::fail_with_message;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool misaligned16(const void *p) { return ((uintptr_t)p & 15) != 0; }

kda_status check_heads(int32_t Hq, int32_t Hkv, int32_t D, kda_dtype dtype)
{
    if (Hq < 1 || Hkv < 1) return fail_with_message(KDA_ERR_INVALID_ARG, "head counts must be >= 1 (got %d, %d)", Hq, Hkv);
    if (Hq % Hkv != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "query heads (%d) not a multiple of key/value heads (%d)", Hq, Hkv);
    if (Hq > 65535) return fail_with_message(KDA_ERR_UNSUPPORTED, "more than 65535 heads");
    if (D != 64 && D != 128) return fail_with_message(KDA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128}", D);
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP32)
        return fail_with_message(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    return KDA_OK;
}

kda_status check_cache(kda_dtype dtype, kda_dtype kv, int32_t page, int32_t cols, int64_t pages, int *shift)
{
    if (kv != dtype && kv != KDA_DTYPE_E4M3)
        return fail_with_message(KDA_ERR_INVALID_ARG, "kv_dtype %d: the cache has the type of q or e4m3", (int)kv);
    if (kv == KDA_DTYPE_E4M3 && dtype != KDA_DTYPE_BF16)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "an e4m3 cache goes with bf16 queries");
    if (page < 16 || page > 1024 || (page & (page - 1)) != 0)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "page_size %d not a power of two in [16, 1024]", page);
    if (cols < 1) return fail_with_message(KDA_ERR_INVALID_ARG, "pages_per_seq must be >= 1 (got %d)", cols);
    if ((int64_t)cols * page > (int64_t)INT32_MAX / 2)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "pages_per_seq x page_size beyond 2^30 tokens");
    if (pages < 0 || pages > INT32_MAX) return fail_with_message(KDA_ERR_INVALID_ARG, "num_pages %lld", (long long)pages);
    *shift = __builtin_ctz((unsigned)page);
    return KDA_OK;
}

struct Layout {
    size_t cu, words, items, joins, ml, parts, total;
    kda::AttnPlan plan;
    int shift;
    bool paged;
};

kda_status check_desc(const kda_attn_desc *d, Layout *lay)
{
    if (!d) return fail_with_message(KDA_ERR_INVALID_ARG, "desc is NULL");
    if (d->num_seqs < 1) return fail_with_message(KDA_ERR_INVALID_ARG, "num_seqs must be >= 1 (got %d)", d->num_seqs);
    if (d->total_tokens < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "total_tokens must be >= 0");
    if (d->total_tokens > (int64_t)INT32_MAX / 2)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "total_tokens %lld too large", (long long)d->total_tokens);
    kda_status s = check_heads(d->num_q_heads, d->num_kv_heads, d->head_dim, d->dtype);
    if (s != KDA_OK) return s;
    if (d->total_tokens * d->num_q_heads > (int64_t)INT32_MAX)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "total_tokens x num_q_heads beyond 2^31");
    if (d->max_seq_len < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "max_seq_len must be >= 0");
    if (!(d->scale >= 0.f) || isinf(d->scale)) return fail_with_message(KDA_ERR_INVALID_ARG, "scale must be finite and >= 0");
    Layout L;
    L.shift = 0;
    L.paged = d->page_size != 0 || d->pages_per_seq != 0 || d->num_pages != 0;
    if (L.paged && (s = check_cache(d->dtype, d->kv_dtype, d->page_size, d->pages_per_seq, d->num_pages, &L.shift)) != KDA_OK)
        return s;
    size_t off = align256(sizeof(kda::DevStatus));   // the status word is first
    L.cu = off; off = align256(off + sizeof(int32_t) * ((size_t)d->num_seqs + 1));
    L.plan = kda::AttnPlan{};
    L.words = L.items = L.joins = L.ml = L.parts = 0;
    if (d->total_tokens > 0 && kda::attn_on_tc(d->dtype)) {
        const int64_t longest = d->max_seq_len > 0 && d->max_seq_len < d->total_tokens ? d->max_seq_len : d->total_tokens;
        L.plan = kda::attn_plan_sizes(d->total_tokens, d->num_seqs, d->num_q_heads, d->num_kv_heads,
                                      L.paged ? (int64_t)d->pages_per_seq * d->page_size : longest);
        L.words = off; off = align256(off + 3 * sizeof(int32_t));
        L.items = off; off = align256(off + (size_t)L.plan.capacity * sizeof(kda::AttnItem));
        L.joins = off; off = align256(off + (size_t)L.plan.slots * sizeof(kda::AttnJoin));
        L.ml = off; off = align256(off + (size_t)L.plan.slots * 256 * sizeof(float2));
        L.parts = off; off = align256(off + (size_t)L.plan.slots * 256 * d->head_dim * sizeof(float));
    }
    L.total = off;
    *lay = L;
    return KDA_OK;
}

struct Cache {
    const void *k, *v;
    const float *ks, *vs;
    const int32_t *table, *lens;
};

// Checks what every attention call has and fills its arguments.
kda_status fill(kda::AttnArgs &a, const void *q, const void *k, const void *v, void *out, float *lse, const kda_attn_desc *d,
                const Layout &L, void *workspace, size_t workspace_bytes, kda_stream_t stream, const Cache *c)
{
    const bool any = d->total_tokens > 0;
    if ((c != nullptr) != L.paged)
        return fail_with_message(KDA_ERR_INVALID_ARG, c ? "desc has no page_size" : "packed keys and values: page_size, pages_per_seq "
                                                                                   "and num_pages must be 0");
    if (any && (!q || !out)) return fail_with_message(KDA_ERR_INVALID_ARG, "q and out must be non-NULL");
    if (any && !c && (!k || !v)) return fail_with_message(KDA_ERR_INVALID_ARG, "k and v must be non-NULL");
    // (a prefill checks the lengths of sequences without a new token too)
    if (c && !c->table != !c->lens) return fail_with_message(KDA_ERR_INVALID_ARG, "page_table and kv_lens go together");
    if (any && c && (!c->table || !c->lens || ((!c->k || !c->v) && d->num_pages > 0)))
        return fail_with_message(KDA_ERR_INVALID_ARG, "k_cache, v_cache, page_table and kv_lens must be non-NULL");
    const bool e4m3 = d->kv_dtype == KDA_DTYPE_E4M3;
    if (c && (e4m3 ? (!c->ks || !c->vs) && d->num_pages > 0 : c->ks || c->vs))
        return fail_with_message(KDA_ERR_INVALID_ARG, "k_scale and v_scale go with an e4m3 cache, and with no other");
    if (!workspace) return fail_with_message(KDA_ERR_WORKSPACE, "workspace is NULL");
    if (workspace_bytes < L.total)
        return fail_with_message(KDA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes, L.total);
    if (((uintptr_t)workspace & 255) != 0) return fail_with_message(KDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (out && (out == q || out == k || out == v || (c && (out == c->k || out == c->v))))
        return fail_with_message(KDA_ERR_INVALID_ARG, "out aliases an input");
    if (misaligned16(q) || misaligned16(k) || misaligned16(v) || misaligned16(out) ||
        (c && (misaligned16(c->k) || misaligned16(c->v) || misaligned16(c->ks) || misaligned16(c->vs))))
        return fail_with_message(KDA_ERR_INVALID_ARG, "q, k, v, out, the cache and its scales must be 16-byte aligned");
    a.q = q; a.k = k; a.v = v; a.cu_seqlens = nullptr; a.out = out; a.lse = lse;
    a.N = d->num_seqs; a.Hq = d->num_q_heads; a.Hkv = d->num_kv_heads; a.D = d->head_dim; a.m = 0; a.T = d->total_tokens;
    a.dtype = d->dtype; a.kv_dtype = c ? d->kv_dtype : d->dtype;
    // (a cache without a page: any address, nothing is read)
    a.kv = c ? kda::PagedKV{c->k ? c->k : q, c->v ? c->v : q, c->ks, c->vs, c->table, c->lens, d->num_pages, d->pages_per_seq, d->page_size, L.shift}
             : kda::PagedKV{};
    a.scale = (float)((d->scale > 0.f ? (double)d->scale : 1.0 / sqrt((double)d->head_dim)) * 1.4426950408889634);
    a.status = nullptr;
    a.plan = kda::AttnPlan{};
    a.cu = (int32_t *)((char *)workspace + L.cu);
    a.wait_limit = d->wait_limit ? d->wait_limit : kda::kDefaultWaitLimit;
    a.bounds = kda::Bounds{a.T - kda::debug_clip_tokens(), 0, 0, 0};
    a.stream = (cudaStream_t)stream;
    return KDA_OK;
}

kda_status prefill(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, void *out, float *lse,
                   const kda_attn_desc *d, void *workspace, size_t workspace_bytes, kda_stream_t stream, const Cache *c)
{
    Layout L;
    kda_status s = check_desc(d, &L);
    if (s != KDA_OK) return s;
    if (!cu_seqlens && d->total_tokens % d->num_seqs != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "total_tokens %lld not a multiple of num_seqs %d (cu_seqlens NULL)",
                                 (long long)d->total_tokens, d->num_seqs);
    kda::AttnArgs a;
    if ((s = fill(a, q, k, v, out, lse, d, L, workspace, workspace_bytes, stream, c)) != KDA_OK) return s;
    a.cu_seqlens = cu_seqlens;
    a.status = &((kda::DevStatus *)workspace)->code;
    const bool tc = a.T > 0 && kda::attn_on_tc(a.dtype);
    if (tc) {
        char *ws = (char *)workspace;
        a.plan = L.plan;
        a.plan.next = (int32_t *)(ws + L.words);
        a.plan.count = a.plan.next + 1;
        a.plan.join_count = a.plan.next + 2;
        a.plan.items = (kda::AttnItem *)(ws + L.items);
        a.plan.joins = (kda::AttnJoin *)(ws + L.joins);
        a.plan.ml = (float2 *)(ws + L.ml);
        a.plan.parts = (float *)(ws + L.parts);
    }
    cudaError_t e = kda::launch_attn_plan(a);
    if (e == cudaSuccess && a.T > 0) e = tc ? kda::launch_attn_tc(a) : kda::launch_attn_f32(a);
    if (e != cudaSuccess) return fail_with_message(KDA_ERR_CUDA, "attention prefill: %s", cudaGetErrorString(e));
    return kda::debug_finish(KDA_OK, a.stream);
}

}  // namespace

extern "C" {

kda_status kda_kv_append(const void *q, const void *k, const void *v, const int32_t *positions, const int32_t *seq_ids,
                         const int32_t *page_table, const float *inv_freq, void *q_out, void *k_out, void *k_cache,
                         void *v_cache, float *k_scale, float *v_scale, int32_t *status, const kda_append_desc *d,
                         kda_stream_t stream)
{
    kda::NvtxRange r("kda_kv_append");
    if (!d) return fail_with_message(KDA_ERR_INVALID_ARG, "desc is NULL");
    const int64_t T = d->total_tokens;
    if (T < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "total_tokens must be >= 0");
    if (T > (int64_t)INT32_MAX / 2) return fail_with_message(KDA_ERR_UNSUPPORTED, "total_tokens %lld too large", (long long)T);
    kda_status s = check_heads(d->num_q_heads, d->num_kv_heads, d->head_dim, d->dtype);
    if (s != KDA_OK) return s;
    const int D = d->head_dim;
    if (d->rotary_dim < 0 || d->rotary_dim > D || d->rotary_dim % 2 != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "rotary_dim %d not even in [0, %d]", d->rotary_dim, D);
    if ((d->rotary_dim > 0) != (inv_freq != nullptr))
        return fail_with_message(KDA_ERR_INVALID_ARG, "inv_freq is given if and only if rotary_dim > 0");
    if (d->interleaved != 0 && d->interleaved != 1) return fail_with_message(KDA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    const bool cache = page_table || k_cache || v_cache;
    int shift = 0;
    if (cache) {
        if (d->num_seqs < 1) return fail_with_message(KDA_ERR_INVALID_ARG, "num_seqs must be >= 1 (got %d)", d->num_seqs);
        if ((s = check_cache(d->dtype, d->kv_dtype, d->page_size, d->pages_per_seq, d->num_pages, &shift)) != KDA_OK) return s;
        if (T > 0 && (!page_table || !k_cache || !v_cache || !seq_ids || !v))
            return fail_with_message(KDA_ERR_INVALID_ARG, "a cache needs page_table, k_cache, v_cache, seq_ids and v");
        if ((d->kv_dtype == KDA_DTYPE_E4M3) != (k_scale && v_scale) || (!k_scale) != (!v_scale))
            return fail_with_message(KDA_ERR_INVALID_ARG, "k_scale and v_scale go with an e4m3 cache, and with no other");
    } else if (k_scale || v_scale) {
        return fail_with_message(KDA_ERR_INVALID_ARG, "scales without a cache");
    }
    if (T > 0 && (!k || !positions)) return fail_with_message(KDA_ERR_INVALID_ARG, "k and positions must be non-NULL");
    if ((q != nullptr) != (q_out != nullptr)) return fail_with_message(KDA_ERR_INVALID_ARG, "q and q_out go together");
    const int64_t piece = d->dtype == KDA_DTYPE_BF16 ? 8 : 4, nq = (int64_t)d->num_q_heads * D, nk = (int64_t)d->num_kv_heads * D;
    const int64_t qs = d->q_stride ? d->q_stride : nq, ks = d->k_stride ? d->k_stride : nk, vs = d->v_stride ? d->v_stride : nk;
    if (qs < nq || ks < nk || vs < nk || qs % piece || ks % piece || vs % piece)
        return fail_with_message(KDA_ERR_INVALID_ARG, "token strides must cover a token's heads and be multiples of 16 bytes");
    if (misaligned16(q) || misaligned16(k) || misaligned16(v) || misaligned16(q_out) || misaligned16(k_out) ||
        misaligned16(k_cache) || misaligned16(v_cache) || misaligned16(k_scale) || misaligned16(v_scale))
        return fail_with_message(KDA_ERR_INVALID_ARG, "q, k, v, q_out, k_out, the cache and its scales must be 16-byte aligned");
    if ((q_out && ((q_out == q && qs != nq) || q_out == k || q_out == v || q_out == k_out)) ||
        (k_out && ((k_out == k && ks != nk) || k_out == v || k_out == q)))
        return fail_with_message(KDA_ERR_INVALID_ARG, "an output aliases an input that it may not be");
    if (T == 0) return KDA_OK;
    const kda::AppendArgs a{q, k, v, positions, seq_ids, page_table, inv_freq, q_out, k_out, k_cache, v_cache, k_scale, v_scale,
                            status, T, d->num_pages, qs, ks, vs, d->num_q_heads, d->num_kv_heads, D, d->rotary_dim,
                            d->interleaved, d->num_seqs, d->pages_per_seq, d->page_size, shift, d->rope_scale, d->dtype,
                            cache ? d->kv_dtype : d->dtype, kda::Bounds{T - kda::debug_clip_tokens(), 0, 0, 0},
                            (cudaStream_t)stream};
    const cudaError_t e = kda::launch_kv_append(a);
    if (e != cudaSuccess) return fail_with_message(KDA_ERR_CUDA, "cache append: %s", cudaGetErrorString(e));
    return kda::debug_finish(KDA_OK, a.stream);
}

size_t kda_attn_workspace_size(const kda_attn_desc *desc)
{
    Layout L;
    return check_desc(desc, &L) == KDA_OK ? L.total : 0;
}

size_t kda_attn_decode_workspace_size(const kda_attn_desc *desc)
{
    Layout L;
    return check_desc(desc, &L) == KDA_OK ? kda::attn_decode_workspace(desc->head_dim) : 0;
}

kda_status kda_attn_prefill(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, void *out, float *lse,
                            const kda_attn_desc *desc, void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    kda::NvtxRange r("kda_attn_prefill");
    return prefill(q, k, v, cu_seqlens, out, lse, desc, workspace, workspace_bytes, stream, nullptr);
}

kda_status kda_attn_prefill_paged(const void *q, const int32_t *cu_seqlens, const void *k_cache, const void *v_cache,
                                  const float *k_scale, const float *v_scale, const int32_t *page_table,
                                  const int32_t *kv_lens, void *out, float *lse, const kda_attn_desc *desc, void *workspace,
                                  size_t workspace_bytes, kda_stream_t stream)
{
    kda::NvtxRange r("kda_attn_prefill_paged");
    const Cache c{k_cache, v_cache, k_scale, v_scale, page_table, kv_lens};
    return prefill(q, nullptr, nullptr, cu_seqlens, out, lse, desc, workspace, workspace_bytes, stream, &c);
}

kda_status kda_attn_decode(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *page_table, const int32_t *kv_lens, void *out, float *lse,
                           const kda_attn_desc *desc, int32_t *status, void *workspace, size_t workspace_bytes,
                           kda_stream_t stream)
{
    kda::NvtxRange r("kda_attn_decode");
    const Cache c{k_cache, v_cache, k_scale, v_scale, page_table, kv_lens};
    Layout L;
    kda_status s = check_desc(desc, &L);
    if (s != KDA_OK) return s;
    L.total = kda::attn_decode_workspace(desc->head_dim);   // (all of it for its parts)
    if (desc->total_tokens % desc->num_seqs != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "total_tokens %lld not a multiple of num_seqs %d",
                                 (long long)desc->total_tokens, desc->num_seqs);
    kda::AttnArgs a;
    if ((s = fill(a, q, nullptr, nullptr, out, lse, desc, L, workspace, workspace_bytes, stream, &c)) != KDA_OK) return s;
    if (a.T == 0) return KDA_OK;
    a.m = (int)(a.T / a.N);
    a.status = status;
    const cudaError_t e = kda::launch_attn_decode(a, workspace);
    if (e != cudaSuccess) return fail_with_message(KDA_ERR_CUDA, "attention decode: %s", cudaGetErrorString(e));
    return kda::debug_finish(KDA_OK, a.stream);
}

}  // extern "C"
