// plan.cu -- kda_plan_batch: the offsets, slot tables and token maps of one
// batch over a state pool, built on the device from request lengths.
//
// A few thousand integers go in and at most some megabytes of token maps come
// out, so the call is bound by latency: one launch, in which every CTA forms
// the prefix sums of the lengths for itself (N <= 16384 of them, in shared
// memory) instead of waiting for another; CTA 0 then assigns the slots while
// the others fill the token maps of their share of the rows by binary search.
#include <atomic>

#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kMaxRequests = 16384;
constexpr int kFillRows = 2048;     // token rows per CTA beyond which more CTAs are used

struct PlanArgs {
    const int32_t *lens, *past, *resume, *slots, *free_slots, *free_head;
    int32_t nfree, N, stride, cols;
    int64_t T, cap;
    int32_t *table, *cu, *init, *slots_out, *ckpt_off, *ckpt, *ids, *pos, *head_out, *status;
};

// Largest n in [0, N) with off[n] <= i.
__device__ __forceinline__ int owner_of(const int32_t *off, int N, int32_t i)
{
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(1024) plan_kernel(PlanArgs a, int64_t rows_per_cta)
{
    extern __shared__ int32_t dyn[];
    __shared__ int64_t sh[32];
    __shared__ int bad_sh, short_sh;
    const int tid = threadIdx.x, NT = blockDim.x, N = a.N;
    int32_t *cu = dyn;                       // [N + 1]
    const bool first_cta = blockIdx.x == 0;
    if (tid == 0) bad_sh = short_sh = 0;

    // offsets of the requests, clamped to the batch's rows; each thread takes a run of requests
    const int run = (N + NT - 1) / NT, n0 = min(N, tid * run), n1 = min(N, n0 + run);
    int64_t mine = 0;
    bool bad = false;
    for (int n = n0; n < n1; ++n) {
        const int32_t L = a.lens[n];
        bad |= L < 0;
        mine += max(L, 0);
    }
    int64_t total;
    int64_t at = block_scan_excl(mine, sh, &total);
    for (int n = n0; n < n1; ++n) {
        cu[n] = (int32_t)min(at, a.T);
        at += max(a.lens[n], 0);
    }
    if (tid == 0) cu[N] = (int32_t)min(total, a.T);
    __syncthreads();

    if (first_cta) {
        int32_t *off = dyn + N + 1, *rank = off + N + 1;   // [N + 1] each: snapshots due before n, slots taken before n
        bad |= total > a.T;
        // snapshots due, and requests that need a state slot
        int64_t due = 0, want = 0;
        for (int n = n0; n < n1; ++n) {
            const int32_t L = cu[n + 1] - cu[n];
            if (a.stride > 0) due += L / a.stride;
            want += a.slots[n] < 0 && L > 0;
        }
        // both counts fit 31 bits (due <= T / 64): one scan of a packed pair
        int64_t tot2;
        const int64_t ex = block_scan_excl((due << 32) | want, sh, &tot2);
        const int32_t dues = (int32_t)(tot2 >> 32), wants = (int32_t)(tot2 & 0xffffffff);
        const int32_t head_in = *a.free_head, head = min(max(head_in, 0), a.nfree);
        bad |= head_in != head;
        int32_t o = (int32_t)(ex >> 32), w = (int32_t)(ex & 0xffffffff);
        bool short_ = false;
        int64_t take = 0;
        for (int n = n0; n < n1; ++n) {
            const int32_t L = cu[n + 1] - cu[n], p_in = a.past ? a.past[n] : 0, p = max(p_in, 0);
            bad |= p_in < 0 || (int64_t)p + L > INT32_MAX;
            const int32_t s = a.slots[n];
            int32_t s_out = s;
            if (s < 0 && L > 0) {
                const int64_t f = (int64_t)head + w++;
                s_out = f < a.nfree ? a.free_slots[f] : -1;
                short_ |= f >= a.nfree;
            }
            const int32_t rs = a.resume ? a.resume[n] : -1;
            a.init[n] = rs >= 0 ? rs : (p > 0 ? max(s, -1) : -1);
            a.slots_out[n] = s_out;
            a.cu[n] = cu[n];
            a.ckpt_off[n] = off[n] = o;
            if (a.stride > 0) {
                const int32_t d = L / a.stride;
                if (p % a.stride == 0) {   // snapshots on the request's grid, as far as the tables reach
                    int64_t t = min((int64_t)d, max((int64_t)0, a.cap - o));
                    if (a.table) t = min(t, max((int64_t)0, (int64_t)a.cols - p / a.stride));
                    take += t;
                }
                o += d;
            }
        }
        if (tid == 0) {
            a.cu[N] = cu[N];
            a.ckpt_off[N] = off[N] = dues;
        }
        int64_t taken;
        int64_t r = block_scan_excl(take, sh, &taken);
        for (int n = n0; n < n1; ++n) {
            rank[n] = (int32_t)r;
            if (a.stride > 0) {
                const int32_t d = (cu[n + 1] - cu[n]) / a.stride, p = a.past ? max(a.past[n], 0) : 0;
                if (p % a.stride == 0) {
                    int64_t t = min((int64_t)d, max((int64_t)0, a.cap - off[n]));
                    if (a.table) t = min(t, max((int64_t)0, (int64_t)a.cols - p / a.stride));
                    r += t;
                }
            }
        }
        if (tid == 0) rank[N] = (int32_t)taken;
        const int64_t base = min((int64_t)head + wants, (int64_t)a.nfree);
        short_ |= base + taken > a.nfree || dues > a.cap;
        if (bad) bad_sh = 1;
        if (short_) short_sh = 1;
        __syncthreads();
        for (int64_t e = tid; e < a.cap; e += NT) {
            int32_t slot = -1;
            if (e < dues) {
                const int n = owner_of(off, N, (int32_t)e);
                const int32_t j = (int32_t)e - off[n];
                const int64_t f = base + rank[n] + j;
                if (j < rank[n + 1] - rank[n] && f < a.nfree) {
                    slot = a.free_slots[f];
                    if (a.table) {
                        const int32_t p = a.past ? max(a.past[n], 0) : 0;
                        a.table[(int64_t)n * a.cols + p / a.stride + j] = slot;
                    }
                }
            }
            a.ckpt[e] = slot;
        }
        if (tid == 0) {
            *a.head_out = (int32_t)min(base + taken, (int64_t)a.nfree);
            if (a.status)
                *a.status = bad_sh ? (int32_t)KDA_ERR_INVALID_ARG : short_sh ? (int32_t)KDA_ERR_CKPT_OVERFLOW : 0;
        }
    }
    // token maps: CTA 0 takes part only when it is alone
    const int64_t fill = gridDim.x == 1 ? 0 : (int64_t)blockIdx.x - 1;
    if (fill < 0) return;
    const int64_t lo = fill * rows_per_cta, hi = min(a.T, lo + rows_per_cta);
    for (int64_t t = lo + tid; t < hi; t += NT) {
        int32_t id = -1, ps = -1;
        if (t < cu[N]) {
            id = owner_of(cu, N, (int32_t)t);
            const int64_t x = (int64_t)(a.past ? max(a.past[id], 0) : 0) + t - cu[id];
            ps = (int32_t)min(x, (int64_t)INT32_MAX);
        }
        a.ids[t] = id;
        a.pos[t] = ps;
    }
}

// The kernel's shared-memory opt-in, once per device.
cudaError_t plan_attributes()
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        if ((e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      3 * (kMaxRequests + 1) * (int)sizeof(int32_t))) != cudaSuccess)
            return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_plan_batch(const int32_t *lens, const int32_t *past, const int32_t *resume_slots,
                                     const int32_t *state_slots, const int32_t *free_slots, int32_t num_free,
                                     const int32_t *free_head, int32_t num_requests, int64_t total_tokens,
                                     int32_t ckpt_stride, int64_t ckpt_capacity, int32_t *snap_table,
                                     int32_t snap_cols, int32_t *cu_seqlens, int32_t *init_slots,
                                     int32_t *state_slots_out, int32_t *ckpt_offsets, int32_t *ckpt_slots,
                                     int32_t *seq_ids, int32_t *positions, int32_t *free_head_out, int32_t *status,
                                     kda_stream_t stream)
{
    using kda::fail_with_message;
    kda::NvtxRange r("kda_plan_batch");
    if (num_requests < 1) return fail_with_message(KDA_ERR_INVALID_ARG, "num_requests must be >= 1 (got %d)", num_requests);
    if (num_requests > kda::kMaxRequests)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "num_requests %d > %d", num_requests, kda::kMaxRequests);
    if (total_tokens < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "total_tokens must be >= 0");
    if (total_tokens > INT32_MAX / 2)
        return fail_with_message(KDA_ERR_UNSUPPORTED, "total_tokens %lld too large", (long long)total_tokens);
    if (ckpt_stride < 0 || ckpt_stride % 64 != 0)
        return fail_with_message(KDA_ERR_INVALID_ARG, "ckpt_stride %d must be 0 or a positive multiple of 64", ckpt_stride);
    if (ckpt_capacity < 0 || ckpt_capacity > INT32_MAX)
        return fail_with_message(KDA_ERR_INVALID_ARG, "ckpt_capacity must be in [0, 2^31)");
    if (num_free < 0) return fail_with_message(KDA_ERR_INVALID_ARG, "num_free must be >= 0");
    if (!lens || !state_slots || !free_head || !cu_seqlens || !init_slots || !state_slots_out || !ckpt_offsets ||
        !free_head_out)
        return fail_with_message(KDA_ERR_INVALID_ARG, "lens, state_slots, free_head and the outputs must be non-NULL");
    if (num_free > 0 && !free_slots) return fail_with_message(KDA_ERR_INVALID_ARG, "free_slots is NULL but num_free > 0");
    if (ckpt_capacity > 0 && !ckpt_slots)
        return fail_with_message(KDA_ERR_INVALID_ARG, "ckpt_slots is NULL but ckpt_capacity > 0");
    if (total_tokens > 0 && (!seq_ids || !positions))
        return fail_with_message(KDA_ERR_INVALID_ARG, "seq_ids and positions must be non-NULL");
    if (snap_cols < 0 || (snap_table && snap_cols == 0))
        return fail_with_message(KDA_ERR_INVALID_ARG, "snap_table needs snap_cols >= 1");
    if (cu_seqlens == lens || init_slots == state_slots || (const int32_t *)init_slots == resume_slots ||
        init_slots == state_slots_out)
        return fail_with_message(KDA_ERR_INVALID_ARG, "an output aliases an input");
    cudaError_t e = kda::plan_attributes();
    if (e != cudaSuccess) return fail_with_message(KDA_ERR_CUDA, "plan kernel: %s", cudaGetErrorString(e));
    const kda::PlanArgs a{lens,         past,     resume_slots, state_slots,     free_slots,   free_head,  num_free,
                          num_requests, ckpt_stride, snap_table ? snap_cols : 0, total_tokens, ckpt_capacity,
                          snap_table,   cu_seqlens, init_slots, state_slots_out, ckpt_offsets, ckpt_slots, seq_ids,
                          positions,    free_head_out, status};
    // one CTA while it can fill the maps by itself, else one for the slots and up to one per other SM
    const int64_t sms = kda::device_sm_count();
    int64_t ctas = 1, rows = total_tokens;
    if (total_tokens > kda::kFillRows) {
        const int64_t fillers = (total_tokens + kda::kFillRows - 1) / kda::kFillRows;
        ctas = 1 + (fillers < sms - 1 ? fillers : sms - 1);
        rows = (total_tokens + ctas - 2) / (ctas - 1);
    }
    const int threads = num_requests <= 256 && total_tokens <= 256 ? 256 : 1024;
    kda::plan_kernel<<<(unsigned)ctas, threads, 3 * ((size_t)num_requests + 1) * sizeof(int32_t), (cudaStream_t)stream>>>(
        a, rows);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return fail_with_message(KDA_ERR_CUDA, "plan kernel: %s", cudaGetErrorString(e));
    return kda::debug_finish(KDA_OK, (cudaStream_t)stream);
}
