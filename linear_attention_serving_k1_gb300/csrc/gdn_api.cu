// gdn_api.cu -- C entry points of the gated delta rule: argument validation,
// workspace layout and kernel dispatch, in the manner of api.cu.
#include <string.h>

#include "gdn.cuh"

namespace {

using kda::fail_with_message;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

kda_status check_dims(int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv, kda_dtype dtype)
{
    if (Hk < 1 || Hv < 1) return fail_with_message(KDA_ERR_INVALID_ARG, "head counts must be >= 1 (got %d, %d)", Hk, Hv);
    if (Hv % Hk != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "value heads (%d) not a multiple of query/key heads (%d)", Hv, Hk);
    if (Dk != 64 && Dk != 128) return fail_with_message(KDA_ERR_UNSUPPORTED, "head_dim_k %d not in {64, 128}", Dk);
    if (Dv < 64 || Dv > 512 || Dv % 64 != 0)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "head_dim_v %d not a multiple of 64 in [64, 512]", Dv);
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP32)
        return fail_with_message(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    return KDA_OK;
}

struct Layout {
    size_t cu, ckpt_off, order, next, carry, offs, trans, total;
    kda::GdnSegs segs;
};

kda_status check_desc(const kda_gdn_desc *d, Layout *lay)
{
    if (!d) return fail_with_message(KDA_ERR_INVALID_ARG, "desc is NULL");
    if (d->num_seqs < 1) return fail_with_message(KDA_ERR_INVALID_ARG, "num_seqs must be >= 1 (got %d)", d->num_seqs);
    if (d->total_tokens < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "total_tokens must be >= 0");
    if (d->total_tokens > (int64_t)INT32_MAX / 2)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "total_tokens %lld too large", (long long)d->total_tokens);
    const kda_status s = check_dims(d->num_qk_heads, d->num_v_heads, d->head_dim_k, d->head_dim_v, d->dtype);
    if (s != KDA_OK) return s;
    if (d->ckpt_stride < 0 || d->ckpt_stride % kda::kGdnChunk != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "ckpt_stride %d must be 0 or a positive multiple of %d", d->ckpt_stride,
                    kda::kGdnChunk);
    if (d->ckpt_capacity < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "ckpt_capacity must be >= 0");
    if (d->max_seq_len < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "max_seq_len must be >= 0");
    // the largest grid: one CTA per sequence, value head and 32 columns
    if ((int64_t)d->num_seqs * d->num_v_heads > INT32_MAX / (d->head_dim_v / 32))
        return fail_with_message(KDA_ERR_UNSUPPORTED, "num_seqs x num_v_heads too large");
    const size_t table = sizeof(int32_t) * ((size_t)d->num_seqs + 1);
    Layout L;
    size_t off = align256(sizeof(kda::DevStatus));   // the status word is first
    L.cu = off; off = align256(off + table);
    L.ckpt_off = off; off = align256(off + table);
    L.order = off; off = align256(off + table);
    L.next = off; off = align256(off + 2 * sizeof(int32_t));
    L.segs = kda::GdnSegs{1, 0, nullptr, nullptr, nullptr};
    if (d->dtype == KDA_DTYPE_BF16 && d->total_tokens > 0) {
        const int64_t bound = d->max_seq_len > 0 && d->max_seq_len < d->total_tokens ? d->max_seq_len : d->total_tokens;
        L.segs = kda::plan_gdn_segs(d->num_seqs, d->num_v_heads, d->head_dim_v, bound);
    }
    const size_t heads = (size_t)d->num_seqs * d->num_v_heads * sizeof(float), P = L.segs.P;
    const size_t state = heads * d->head_dim_k * d->head_dim_v, square = heads * d->head_dim_k * d->head_dim_k;
    L.carry = off; off = align256(off + (P > 1 ? P - 1 : 0) * state);
    L.offs = off; off = align256(off + (P > 2 ? P - 2 : 0) * state);
    L.trans = off; off = align256(off + (P > 2 ? P - 2 : 0) * square);
    L.total = off;
    *lay = L;
    return KDA_OK;
}

bool misaligned16(const void *p) { return ((uintptr_t)p & 15) != 0; }

kda_status prefill(const void *q, const void *k, const void *v, const float *g, const float *beta,
                   const float *init_state, const int32_t *cu_seqlens, void *out, float *final_state, float *ckpts,
                   const kda_gdn_desc *desc, void *workspace, size_t workspace_bytes, kda_stream_t stream,
                   const kda::PoolArgs *pool)
{
    Layout L;
    kda_status s = check_desc(desc, &L);
    if (s != KDA_OK) return s;
    const int64_t T = desc->total_tokens;
    if (T > 0 && (!q || !k || !v || !g || !beta || !out))
        return fail_with_message(KDA_ERR_INVALID_ARG, "q, k, v, g, beta and out must be non-NULL");
    if (!cu_seqlens && T % desc->num_seqs != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "total_tokens %lld not a multiple of num_seqs %d (cu_seqlens NULL)",
                    (long long)T, desc->num_seqs);
    if (pool) {
        if (pool->slots < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "pool_slots must be >= 0");
        if (!pool->pool && (pool->init_slots || pool->final_slots || pool->ckpt_slots))
            return fail_with_message(KDA_ERR_INVALID_ARG, "state_pool is NULL but a slot table is given");
        if (desc->ckpt_stride > 0 && desc->ckpt_capacity > 0 && !pool->ckpt_slots)
            return fail_with_message(KDA_ERR_INVALID_ARG, "ckpt_slots is NULL but ckpt_capacity > 0");
        if (misaligned16(pool->pool)) return fail_with_message(KDA_ERR_INVALID_ARG, "state_pool must be 16-byte aligned");
    } else {
        if (desc->ckpt_stride > 0 && !ckpts && desc->ckpt_capacity > 0)
            return fail_with_message(KDA_ERR_INVALID_ARG, "ckpts is NULL but ckpt_capacity > 0");
        if (misaligned16(init_state) || misaligned16(final_state) || misaligned16(ckpts))
            return fail_with_message(KDA_ERR_INVALID_ARG, "states and checkpoints must be 16-byte aligned");
    }
    if (!workspace) return fail_with_message(KDA_ERR_WORKSPACE, "workspace is NULL");
    if (workspace_bytes < L.total)
        return fail_with_message(KDA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes, L.total);
    if (((uintptr_t)workspace & 255) != 0)
        return fail_with_message(KDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (out && (out == q || out == k || out == v))
        return fail_with_message(KDA_ERR_INVALID_ARG, "out aliases an input");
    if (misaligned16(q) || misaligned16(k) || misaligned16(v) || misaligned16(out))
        return fail_with_message(KDA_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");

    char *ws = (char *)workspace;
    kda::GdnArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.cu_seqlens = cu_seqlens; a.out = out;
    a.N = desc->num_seqs; a.Hk = desc->num_qk_heads; a.Hv = desc->num_v_heads;
    a.Dk = desc->head_dim_k; a.Dv = desc->head_dim_v; a.T = T; a.dtype = desc->dtype;
    const int stride = desc->ckpt_stride;
    if (pool)   // every state lives in the pool; a NULL table means none of that kind
        a.io = kda::StateIO{pool->init_slots ? pool->pool : nullptr, pool->final_slots ? pool->pool : nullptr,
                            stride > 0 && pool->ckpt_slots ? pool->pool : nullptr, pool->init_slots, pool->final_slots,
                            pool->ckpt_slots, pool->slots, desc->ckpt_capacity, stride};
    else
        a.io = kda::StateIO{init_state, final_state, stride > 0 ? ckpts : nullptr, nullptr, nullptr, nullptr, 0,
                            desc->ckpt_capacity, stride};
    a.status = (kda::DevStatus *)ws;
    a.tab = kda::GdnTable{(int32_t *)(ws + L.cu), (int32_t *)(ws + L.ckpt_off), (int32_t *)(ws + L.order),
                          (int32_t *)(ws + L.next), cu_seqlens, T, desc->ckpt_capacity, a.N, stride};
    a.segs = L.segs;
    a.segs.carry = (float *)(ws + L.carry);
    a.segs.offs = (float *)(ws + L.offs);
    a.segs.trans = (float *)(ws + L.trans);
    a.wait_limit = desc->wait_limit ? desc->wait_limit : kda::kDefaultWaitLimit;
    a.bounds = kda::Bounds{T - kda::debug_clip_tokens(), 0, pool ? pool->slots : a.N,
                           pool ? pool->slots : desc->ckpt_capacity};
    a.stream = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    const bool chunked = a.dtype == KDA_DTYPE_BF16 && T > 0;
    if (!kda::gdn_few(a)) {
        e = kda::launch_gdn_table(a);
    } else {
        a.tab.cu = nullptr;
        // (the kernel token by token, which waits for nothing, has one writer of the status)
        if (chunked) e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), a.stream);
    }
    if (e == cudaSuccess) e = chunked ? kda::launch_gdn_tc(a) : kda::launch_gdn_scan(a);
    if (e != cudaSuccess) return fail_with_message(KDA_ERR_CUDA, "gated delta rule prefill: %s", cudaGetErrorString(e));
    return kda::debug_finish(KDA_OK, a.stream);
}

kda_status decode(const void *q, const void *k, const void *v, const float *g, const float *beta, float *state,
                  int64_t pool_slots, const int32_t *slot_ids, const int32_t *commit, void *out, int32_t N, int32_t m,
                  int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv, kda_dtype dtype, int32_t *status,
                  kda_stream_t stream)
{
    if (N < 0 || m < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "N and m must be >= 0");
    const kda_status s = check_dims(Hk, Hv, Dk, Dv, dtype);
    if (s != KDA_OK) return s;
    if (slot_ids && pool_slots < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "pool_slots must be >= 0");
    if ((int64_t)N * Hv > INT32_MAX / (Dv / 32) || (int64_t)N * m > INT32_MAX)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "N x m x Hv too large");
    if ((int64_t)N * m == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !state || !out)
        return fail_with_message(KDA_ERR_INVALID_ARG, "q, k, v, g, beta, state and out must be non-NULL");
    if (misaligned16(state)) return fail_with_message(KDA_ERR_INVALID_ARG, "state must be 16-byte aligned");
    if (out == q || out == k || out == v || out == (void *)state)
        return fail_with_message(KDA_ERR_INVALID_ARG, "out aliases an input");
    const kda::GdnDecodeArgs a{q, k, v, g, beta, state, slot_ids, pool_slots, commit, out, N, m, Hk, Hv, Dk, Dv, dtype,
                               slot_ids ? status : nullptr,
                               kda::Bounds{(int64_t)N * m - kda::debug_clip_tokens(), 0, slot_ids ? pool_slots : N, 0},
                               (cudaStream_t)stream};
    const cudaError_t e = kda::launch_gdn_decode(a);
    if (e != cudaSuccess) return fail_with_message(KDA_ERR_CUDA, "gated delta rule decode: %s", cudaGetErrorString(e));
    return kda::debug_finish(KDA_OK, (cudaStream_t)stream);
}

}  // namespace

extern "C" {

size_t kda_gdn_workspace_size(const kda_gdn_desc *desc)
{
    Layout L;
    return check_desc(desc, &L) == KDA_OK ? L.total : 0;
}

kda_status kda_gdn_prefill(const void *q, const void *k, const void *v, const float *g, const float *beta,
                           const float *init_state, const int32_t *cu_seqlens, void *out, float *final_state,
                           float *ckpts, const kda_gdn_desc *desc, void *workspace, size_t workspace_bytes,
                           kda_stream_t stream)
{
    kda::NvtxRange r("kda_gdn_prefill");
    return prefill(q, k, v, g, beta, init_state, cu_seqlens, out, final_state, ckpts, desc, workspace, workspace_bytes,
                   stream, nullptr);
}

kda_status kda_gdn_prefill_pooled(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                  const int32_t *cu_seqlens, void *out, float *state_pool, int64_t pool_slots,
                                  const int32_t *init_slots, const int32_t *final_slots, const int32_t *ckpt_slots,
                                  const kda_gdn_desc *desc, void *workspace, size_t workspace_bytes,
                                  kda_stream_t stream)
{
    kda::NvtxRange r("kda_gdn_prefill_pooled");
    const kda::PoolArgs pool{state_pool, pool_slots, init_slots, final_slots, ckpt_slots};
    return prefill(q, k, v, g, beta, nullptr, cu_seqlens, out, nullptr, nullptr, desc, workspace, workspace_bytes,
                   stream, &pool);
}

kda_status kda_gdn_decode(const void *q, const void *k, const void *v, const float *g, const float *beta, float *state,
                          int64_t pool_slots, const int32_t *slot_ids, void *out, int32_t N, int32_t Hk, int32_t Hv,
                          int32_t Dk, int32_t Dv, kda_dtype dtype, int32_t *status, kda_stream_t stream)
{
    kda::NvtxRange r("kda_gdn_decode");
    return decode(q, k, v, g, beta, state, pool_slots, slot_ids, nullptr, out, N, 1, Hk, Hv, Dk, Dv, dtype, status,
                  stream);
}

kda_status kda_gdn_decode_multi(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                float *state, int64_t pool_slots, const int32_t *slot_ids, const int32_t *commit_len,
                                void *out, int32_t N, int32_t m, int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv,
                                kda_dtype dtype, int32_t *status, kda_stream_t stream)
{
    kda::NvtxRange r("kda_gdn_decode_multi");
    return decode(q, k, v, g, beta, state, pool_slots, slot_ids, commit_len, out, N, m, Hk, Hv, Dk, Dv, dtype, status,
                  stream);
}

}  // extern "C"
