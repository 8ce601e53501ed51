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
};

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

// Sequence table of a call (one launch; also clears the status word).
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
