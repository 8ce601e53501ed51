// gdn.cuh -- the gated delta rule's internal interface between its C entry
// points (gdn_api.cu) and its kernels (gdn_scan.cu, gdn_tc.cu, gdn_decode.cu).
#pragma once

#include "kda_common.cuh"

namespace kda {

// Token offsets, first checkpoint slots and a processing order (longest
// sequences first) of a call, built on the device from cu_seqlens.
struct GdnTable {
    int32_t *cu;         // [N + 1] validated copy (all zero when cu_seqlens is malformed)
    int32_t *ckpt_off;   // [N + 1]
    int32_t *order;      // [N]
    int32_t *next;       // [2] chains handed out so far (the chunked kernel's CTAs, in each of two passes)
    // a call of up to kGdnFew sequences whose CTAs all run at once needs neither an order
    // nor a counter: cu is NULL then, and every CTA reads the offsets for itself, which
    // saves the launch of the table (2 us of host time, 4 us of the GPU's)
    const int32_t *raw;          // cu_seqlens (NULL: equal lengths)
    int64_t T, capacity;
    int N, stride;
};

constexpr int kGdnFew = 31;      // N + 1 offsets in a warp

// One sequence: its number, first row, length and first checkpoint slot.
struct GdnSeq {
    int n, t0, len, ckpt;
};

// The sequence at place `at` of the table's order, or sequence `at` of a call without
// a table (then all lanes of a warp call this, and a status given is set: stored if
// nothing else of the launch reports to it, else recorded beside what the others
// report, on a word that was cleared before the launch).
template <bool SOLE = true>
__device__ __forceinline__ GdnSeq gdn_sequence(const GdnTable &tab, int at, DevStatus *st)
{
    if (tab.cu) {
        const int n = tab.order[at], t0 = tab.cu[n];
        return {n, t0, tab.cu[n + 1] - t0, tab.ckpt_off[n]};
    }
    const int lane = threadIdx.x & 31, N = tab.N;
    const int32_t x = lane > N ? 0 : tab.raw ? tab.raw[lane] : (int32_t)(tab.T / N) * lane;
    // (offsets are compared, not their differences, which may wrap: in order from 0 to at most T
    // they and the lengths are all within [0, T])
    const int32_t next = __shfl_down_sync(0xffffffffu, x, 1);
    const bool bad = (lane < N && next < x) || (lane == 0 && x != 0) || (lane == N && x > tab.T);
    const bool ok = !__any_sync(0xffffffffu, bad);
    const int32_t len = ok && lane < N ? next - x : 0;
    const int32_t cks = tab.stride > 0 ? len / tab.stride : 0;
    int32_t upto = cks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (st && lane == 31) {
        const int32_t code = !ok ? (int32_t)KDA_ERR_INVALID_ARG
                                 : (tab.stride > 0 && upto > tab.capacity) ? (int32_t)KDA_ERR_CKPT_OVERFLOW : 0;
        if (SOLE) st->code = code;
        else if (code != 0) record_status(st, code);
    }
    const int t0 = __shfl_sync(0xffffffffu, x, at), l = __shfl_sync(0xffffffffu, len, at);
    return {at, ok ? t0 : 0, l, __shfl_sync(0xffffffffu, upto - cks, at)};
}

// Few, long chains: every sequence in up to P segments of G chunks (the last
// takes the rest), in two passes with a join between them (gdn_tc.cu); P = 1:
// one pass.  All in the workspace, blocks [N, Hv] each.
struct GdnSegs {
    int P, G;
    float *carry;        // [P - 1][N, Hv, Dk, Dv] state that segment p + 1 starts from
    float *offs;         // [P - 2][N, Hv, Dk, Dv] end state of segment p + 1 started from zeros
    float *trans;        // [P - 2][N, Hv, Dk, Dk] its transition matrix
};

struct GdnArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    const int32_t *cu_seqlens;   // may be NULL
    void *out;
    int N, Hk, Hv, Dk, Dv;
    int64_t T;
    kda_dtype dtype;
    StateIO io;
    DevStatus *status;
    GdnTable tab;
    GdnSegs segs;
    uint32_t wait_limit;
    Bounds bounds;
    cudaStream_t stream;
};

constexpr int kGdnChunk = 64;

// Whether a call goes without the table's launch; the table (one launch; also sets the
// status word).
bool gdn_few(const GdnArgs &a);
cudaError_t launch_gdn_table(const GdnArgs &a);
// Token by token on the CUDA cores, any dtype.
cudaError_t launch_gdn_scan(const GdnArgs &a);
// In chunks on the tensor cores, bf16, T > 0; its segments (P, G) for a call of
// that shape whose longest sequence has up to max_len tokens.
cudaError_t launch_gdn_tc(const GdnArgs &a);
GdnSegs plan_gdn_segs(int64_t N, int64_t Hv, int Dv, int64_t max_len);

struct GdnDecodeArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    float *state;
    const int32_t *slots;        // NULL: dense states
    int64_t pool;
    const int32_t *commit;       // NULL: every token
    void *out;
    int N, m, Hk, Hv, Dk, Dv;
    kda_dtype dtype;
    int32_t *status;
    Bounds bounds;
    cudaStream_t stream;
};
cudaError_t launch_gdn_decode(const GdnDecodeArgs &a);

}  // namespace kda
