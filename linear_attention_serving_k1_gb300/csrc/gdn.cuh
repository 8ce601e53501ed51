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
    int32_t *next;       // chains handed out so far (the chunked kernel's CTAs)
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
    uint32_t wait_limit;
    Bounds bounds;
    cudaStream_t stream;
};

constexpr int kGdnChunk = 64;

// Sequence table of a call (one launch; also clears the status word).
cudaError_t launch_gdn_table(const GdnArgs &a);
// Token by token on the CUDA cores, any dtype.
cudaError_t launch_gdn_scan(const GdnArgs &a);
// In chunks on the tensor cores, bf16, T > 0.
cudaError_t launch_gdn_tc(const GdnArgs &a);

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
