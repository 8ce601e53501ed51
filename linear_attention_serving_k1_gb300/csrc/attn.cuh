// attn.cuh -- the attention layers' internal interface between their C entry
// points (attn_api.cu) and their kernels (kv_append.cu, attn_plan.cu, attn_tc.cu,
// attn_f32.cu, attn_decode.cu), and what those share: the paged cache and the query rows of a sequence.
#pragma once

#include "kda_common.cuh"

namespace kda {

// A paged cache: elements [num_pages, Hkv, page, D], table [N, cols].
struct PagedKV {
    const void *k, *v;
    const float *ks, *vs;        // scales of an e4m3 cache, else NULL
    const int32_t *table;        // NULL: packed keys and values [T, Hkv, D]
    const int32_t *lens;         // [N] tokens of each sequence
    int64_t pages;
    int cols, page, shift;       // page = 1 << shift
};

// A kernel that may be set up while the one before it in the stream still runs: it waits
// for that one's results itself (after_previous, every CTA, before it reads any), and that one
// says, at its start, that its follower may come (next_may_start).
template <typename... P, typename... A>
cudaError_t launch_following(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Number of a sequence's page that holds position p (within the table), -1 if it names none.
__device__ __forceinline__ int64_t page_of(const PagedKV &c, int64_t n, int p)
{
    const int32_t g = c.table[n * c.cols + (p >> c.shift)];
    return g >= 0 && g < c.pages ? g : -1;
}

// Tokens of sequence n, within what its table can hold; *bad: it said otherwise.
__device__ __forceinline__ int kv_length(const PagedKV &c, int64_t n, bool *bad)
{
    const int64_t most = (int64_t)c.cols << c.shift, len = c.lens[n];
    *bad = len < 0 || len > most;
    return (int)(len < 0 ? 0 : len > most ? most : len);
}

// A prefill's work on the tensor cores: blocks of queries, and steps of 128 keys of each.
struct AttnItem {
    int32_t n, block, kt0, kt1, slot;   // slot: of a part of the keys, -1: all of them
};
struct AttnJoin {                       // an item that was cut: its parts' first slot and number
    int32_t n, block, slot, parts;
};
struct AttnPlan {
    int two_heads;               // an item's two tiles: two heads of a block of 128 queries, or a block of 256
    int pairs;                   // items of a block
    int split;                   // whether items may be cut along the keys
    int64_t capacity, slots;     // items; parts of items of one pair each
    int32_t *next, *count, *join_count;
    AttnItem *items;             // longest first
    AttnJoin *joins;
    float *parts;                // [slots][2][128][D]
    float2 *ml;                  // [slots][2][128] maximum, sum
};

struct AttnArgs {
    const void *q, *k, *v;       // k, v: packed keys and values (kv.table NULL)
    const int32_t *cu_seqlens;   // may be NULL
    void *out;
    float *lse;                  // may be NULL
    int N, Hq, Hkv, D, m;        // m: tokens a sequence of a decode call, 0 for a prefill
    int64_t T;
    kda_dtype dtype, kv_dtype;
    PagedKV kv;
    float scale;                 // of the scores, times log2 e
    int32_t *status;             // may be NULL (decode)
    int32_t *cu;                 // validated copy of cu_seqlens (prefill)
    AttnPlan plan;               // prefill on the tensor cores
    uint32_t wait_limit;
    Bounds bounds;
    cudaStream_t stream;
};

// Validates cu_seqlens into a.cu (all zero when malformed), sets the status word and, for
// the tensor cores, lists the items.
cudaError_t launch_attn_plan(const AttnArgs &a);
// Whether a call runs on the tensor cores, and what its plan holds but for the addresses
// (keys: that a sequence may have).
bool attn_on_tc(kda_dtype dtype);
AttnPlan attn_plan_sizes(int64_t T, int64_t N, int Hq, int Hkv, int64_t keys);
cudaError_t launch_attn_tc(const AttnArgs &a);
// Prefill in fp32.
cudaError_t launch_attn_f32(const AttnArgs &a);
// Decode: m > 0 tokens a sequence over the cache; the workspace it takes for parts.
cudaError_t launch_attn_decode(const AttnArgs &a, void *workspace);
size_t attn_decode_workspace(int D);

struct AppendArgs {
    const void *q, *k, *v;
    const int32_t *positions, *seq_ids, *table;
    const float *inv_freq;
    void *q_out, *k_out, *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int32_t *status;
    int64_t T, pages, qs, ks, vs;   // qs, ks, vs: elements from a token to the next
    int Hq, Hkv, D, R, interleaved, N, cols, page, shift;
    float rope_scale;
    kda_dtype dtype, kv_dtype;
    Bounds bounds;
    cudaStream_t stream;
};
cudaError_t launch_kv_append(const AppendArgs &a);

DbgWord dbg_take_attn_f32();
DbgWord dbg_take_attn_tc();
DbgWord dbg_take_attn_decode();
DbgWord dbg_take_kv_append();

}  // namespace kda
