// attn_plan.cu -- the table of a prefill: token offsets, checked, and the items of the
// tensor-core kernel, longest first.
//
// One CTA.  The items are sorted by a counting sort over the number of their steps
// (scaled to 1024 counters); the order among equals is that of the atomics, on which no
// result depends.  Where a call is small (AttnPlan::split), items are cut into equal parts
// of at most s steps, s being the one of 32 lengths about an SM's share of all steps (each
// warp tries one) with the shortest estimate: the rounds that the parts longer than s / 2
// take, or all steps shared evenly if that is longer; a part costs 3 steps more (its start
// and end, and the join).  A plain share instead cut 16 items of 1024 steps into 160
// parts for 152 SMs, which took two rounds (528 us, one round of 144 parts 290).
#include "attn.cuh"

namespace kda {
namespace {

constexpr int kThreads = 1024, kBuckets = 1024;

struct Args {
    const int32_t *raw;
    int32_t *cu, *status;
    int N, items;        // items: whether they are wanted
    int64_t T;
    PagedKV kv;
    AttnPlan plan;
    int sms;
};

__global__ void __launch_bounds__(kThreads) attn_plan_kernel(const Args a)
{
    __shared__ int64_t sh[kThreads / 32];
    __shared__ int sh_i[kThreads / 32], count[kBuckets], sh_max, sh_join, sh_slot;
    __shared__ unsigned long long sh_best;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    // (offsets are compared, not their differences, which may wrap)
    bool bad = false;
    for (int i = tid; i <= a.N; i += blockDim.x) {
        const int32_t x = a.raw ? a.raw[i] : (int32_t)(a.T / a.N) * i;
        bad = bad || x < 0 || x > a.T || (i == 0 && x != 0) || (i > 0 && a.raw && x < a.raw[i - 1]);
    }
    const bool any = __syncthreads_or(bad);
    for (int i = tid; i <= a.N; i += blockDim.x) a.cu[i] = any ? 0 : a.raw ? a.raw[i] : (int32_t)(a.T / a.N) * i;
    if (tid == 0) {
        *a.status = any ? (int32_t)KDA_ERR_INVALID_ARG : 0;
        if (a.items) *a.plan.next = *a.plan.count = *a.plan.join_count = 0;
        sh_max = sh_join = sh_slot = 0;
        sh_best = (1ull << 62) | (1 << 30);
    }
    if (!a.items || any) return;
    for (int i = tid; i < kBuckets; i += blockDim.x) count[i] = 0;
    __syncthreads();
    // f(n, block, steps) of every block of queries: a warp a sequence, a lane a block
    const int rows = a.plan.two_heads ? 128 : 256;
    auto each = [&](auto f) {
        for (int n = warp; n < a.N; n += warps) {
            const int len = a.cu[n + 1] - a.cu[n];
            bool off = false;
            const int total = a.kv.table ? kv_length(a.kv, n, &off) : len;
            if (off && lane == 0) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
            for (int b = lane; b < (len + rows - 1) / rows; b += 32) {
                const int end = total - len + min(len, (b + 1) * rows);
                f(n, b, end > 128 ? (end + 127) / 128 : 1);
            }
        }
    };
    int64_t mine = 0, units;
    int longest = 0;
    each([&](int, int, int t) {
        mine += t;
        longest = max(longest, t);
    });
    block_scan_excl<int64_t>(mine, sh, &units);
    atomicMax(&sh_max, longest);
    __syncthreads();
    int share = 1 << 30;                         // (more steps than any item has: none is cut)
    auto cut = [&](int t, int s, int *parts) {   // steps of a part
        *parts = (t + s - 1) / s;
        return (t + *parts - 1) / *parts;
    };
    if (a.plan.split) {
        constexpr int kExtra = 3, kLeast = 4;
        const int64_t all = units * a.plan.pairs;
        // 0.9 to 2.2 times the share, or no cut
        const double want = (double)all / a.sms * 0.9 * exp2(warp * (1.3 / 30));
        const int s = warp == 31 ? 1 << 30 : want < kLeast ? kLeast : want > 1e8 ? 100000000 : (int)ceil(want);
        int64_t parts = 0, large = 0, slots = 0;
        const int limit = warp == 31 ? sh_max : s;   // steps of the longest part
        int top = 0;
        for (int n = 0; n < a.N; ++n) {              // (all warps over all sequences: calls that may be cut are small)
            const int len = a.cu[n + 1] - a.cu[n];
            bool off = false;
            const int total = a.kv.table ? kv_length(a.kv, n, &off) : len;
            for (int b = lane; b < (len + rows - 1) / rows; b += 32) {
                const int end = total - len + min(len, (b + 1) * rows), t = end > 128 ? (end + 127) / 128 : 1;
                int c;
                const int each_s = cut(t, s, &c);
                parts += c;
                top = max(top, each_s);
                if (each_s > limit / 2) large += c;
                if (c > 1) slots += c;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            parts += __shfl_xor_sync(0xffffffffu, parts, o);
            large += __shfl_xor_sync(0xffffffffu, large, o);
            slots += __shfl_xor_sync(0xffffffffu, slots, o);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        parts *= a.plan.pairs;
        large *= a.plan.pairs;
        const int64_t rounds = (large + a.sms - 1) / a.sms, by_rounds = rounds * (top + kExtra),
                      by_steps = (all + kExtra * parts + a.sms - 1) / a.sms;
        const int64_t cost = by_rounds > by_steps ? by_rounds : by_steps;
        if (lane == 0 && slots * a.plan.pairs <= a.plan.slots)
            atomicMin(&sh_best, ((unsigned long long)cost << 32) | (unsigned)s);
        __syncthreads();
        share = (int)(unsigned)sh_best;
    }
    int shift = 0;
    while (sh_max >> shift >= kBuckets) ++shift;
    each([&](int, int, int t) {
        int parts;
        const int s = cut(t, share, &parts);
        atomicAdd(&count[kBuckets - 1 - (s >> shift)], parts);
    });
    __syncthreads();
    int all = 0;
    const int x = tid < kBuckets ? count[tid] : 0, at = block_scan_excl<int>(x, sh_i, &all);
    if (tid < kBuckets) count[tid] = at;
    if (tid == 0) *a.plan.count = all;
    __syncthreads();
    each([&](int n, int b, int t) {
        int parts;
        const int s = cut(t, share, &parts);
        int slot = -1;
        if (parts > 1) {
            slot = atomicAdd(&sh_slot, parts);
            a.plan.joins[atomicAdd(&sh_join, 1)] = AttnJoin{n, b, slot, parts};
        }
        const int place = atomicAdd(&count[kBuckets - 1 - (s >> shift)], parts);
        for (int i = 0; i < parts; ++i)
            a.plan.items[place + i] = AttnItem{n, b, min(t, i * s), min(t, (i + 1) * s), parts > 1 ? slot + i : -1};
    });
    __syncthreads();
    if (tid == 0) *a.plan.join_count = sh_join;
}

}  // namespace

AttnPlan attn_plan_sizes(int64_t T, int64_t N, int Hq, int Hkv)
{
    AttnPlan p = {};
    p.two_heads = Hq / Hkv % 2 == 0;
    p.pairs = p.two_heads ? Hq / 2 : Hq;
    const int64_t rows = p.two_heads ? 128 : 256, sms = device_sm_count();
    // with four items an SM, longest first, the last ones leave no SM idle for long
    p.split = (T + rows - 1) / rows * p.pairs < 4 * sms;
    p.slots = p.split ? 2 * sms : 0;
    p.capacity = T / rows + N + p.slots;
    return p;
}

cudaError_t launch_attn_plan(const AttnArgs &a)
{
    const bool items = a.plan.items != nullptr;
    const Args x{a.cu_seqlens, a.cu, a.status, a.N, items, a.T, a.kv, a.plan, (int)device_sm_count()};
    attn_plan_kernel<<<1, kThreads, 0, a.stream>>>(x);
    return cudaGetLastError();
}

}  // namespace kda
