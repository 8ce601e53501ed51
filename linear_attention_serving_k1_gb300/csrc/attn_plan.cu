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
// parts for 152 SMs, which took two rounds (528 us, one round of 144 parts 360).
#include "attn.cuh"

namespace kda {
namespace {

constexpr int kThreads = 1024, kBuckets = 1024, kPlanCached = 2048;
static_assert(kThreads == kBuckets, "a counter a thread");

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
    __shared__ int2 seqs[kPlanCached];           // new tokens, all tokens of a sequence
    __shared__ unsigned long long sh_best;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreads / 32;
    next_may_start();
    // (offsets are compared, not their differences, which may wrap)
    bool bad = false, off = false;
    const int32_t equal = (int32_t)(a.T / a.N);
    for (int i = tid; i <= a.N; i += kThreads) {
        const int32_t x = a.raw ? a.raw[i] : equal * i, next = i == a.N ? x : a.raw ? a.raw[i + 1] : equal * (i + 1);
        bad = bad || x < 0 || x > a.T || (i == 0 && x != 0) || next < x;
        if (i == a.N) break;
        bool o = false;
        const int total = a.kv.table ? kv_length(a.kv, i, &o) : next - x;
        off = off || o;
        if (i < kPlanCached) seqs[i] = make_int2(next - x, total);
    }
    for (int i = tid; i < kBuckets; i += kThreads) count[i] = 0;
    if (tid == 0) {
        if (a.items) *a.plan.next = *a.plan.count = *a.plan.join_count = 0;
        sh_max = sh_join = sh_slot = 0;
        sh_best = (1ull << 62) | (1 << 30);
    }
    const bool any = __syncthreads_or(bad), any_off = __syncthreads_or(off);
    if (tid == 0) *a.status = any || any_off ? (int32_t)KDA_ERR_INVALID_ARG : 0;
    for (int i = tid; i <= a.N; i += kThreads) a.cu[i] = any ? 0 : a.raw ? a.raw[i] : equal * i;
    if (!a.items || any) return;
    const int rows = a.plan.two_heads ? 128 : 256;
    auto seq = [&](int n) -> int2 {
        if (n < kPlanCached) return seqs[n];
        const int len = a.raw ? a.raw[n + 1] - a.raw[n] : equal;
        bool o;
        return make_int2(len, a.kv.table ? kv_length(a.kv, n, &o) : len);
    };
    // f(n, block, steps) of every block of queries: of `ws` warps, warp w a sequence and its lanes
    // the blocks, or, of many sequences, a lane each
    auto each = [&](int w, int ws, auto f) {
        const bool many = a.N >= 4 * ws;
        for (int n = many ? w * 32 + lane : w; n < a.N; n += many ? ws * 32 : ws) {
            const int2 x = seq(n);
            const int blocks = (x.x + rows - 1) / rows;
            for (int b = many ? 0 : lane; b < blocks; b += many ? 1 : 32) {
                const int end = x.y - x.x + min(x.x, (b + 1) * rows);
                f(n, b, end > 128 ? (end + 127) / 128 : 1);
            }
        }
    };
    int64_t mine = 0, units;
    int longest = 0;
    each(warp, kWarps, [&](int, int, int t) {
        mine += t;
        longest = max(longest, t);
    });
    block_scan_excl<int64_t>(mine, sh, &units);
    atomicMax(&sh_max, longest);
    __syncthreads();
    int share = 1 << 30;                         // (more steps than any item has: none is cut)
    auto cut = [&](int t, int s, int *parts) {   // steps of a part
        *parts = t <= s ? 1 : (t + s - 1) / s;
        return t <= s ? t : (t + *parts - 1) / *parts;
    };
    if (a.plan.split) {
        constexpr int kExtra = 3, kLeast = 4;
        const float all = (float)units * (float)a.plan.pairs;
        // 0.9 to 2.2 times the share, or no cut
        const float want = all / (float)a.sms * 0.9f * exp2f((float)warp * (1.3f / 30));
        const int s = warp == 31 ? 1 << 30 : want < kLeast ? kLeast : want > 1e8f ? 100000000 : (int)ceilf(want);
        const int half = (warp == 31 ? sh_max : s) / 2;
        int parts = 0, large = 0, slots = 0, top = 0;
        each(0, 1, [&](int, int, int t) {
            int c;
            const int steps = cut(t, s, &c);
            parts += c;
            top = max(top, steps);
            if (steps > half) large += c;
            if (c > 1) slots += c;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            parts += __shfl_xor_sync(0xffffffffu, parts, o);
            large += __shfl_xor_sync(0xffffffffu, large, o);
            slots += __shfl_xor_sync(0xffffffffu, slots, o);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        const float pairs = (float)a.plan.pairs, rounds = ceilf((float)large * pairs / (float)a.sms);
        const float by_rounds = rounds * (float)(top + kExtra), by_steps = (all + kExtra * pairs * (float)parts) / (float)a.sms;
        if (lane == 0 && (int64_t)slots * a.plan.pairs <= a.plan.slots)
            atomicMin(&sh_best, ((unsigned long long)(8.f * fmaxf(by_rounds, by_steps)) << 32) | (unsigned)s);
        __syncthreads();
        share = (int)(unsigned)sh_best;
    }
    int shift = 0;
    while (sh_max >> shift >= kBuckets) ++shift;
    each(warp, kWarps, [&](int, int, int t) {
        int parts;
        const int s = cut(t, share, &parts);
        atomicAdd(&count[kBuckets - 1 - (s >> shift)], parts);
    });
    __syncthreads();
    int all = 0;
    const int x = count[tid], at = block_scan_excl<int>(x, sh_i, &all);
    count[tid] = at;
    if (tid == 0) *a.plan.count = all;
    __syncthreads();
    each(warp, kWarps, [&](int n, int b, int t) {
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

AttnPlan attn_plan_sizes(int64_t T, int64_t N, int Hq, int Hkv, int64_t keys)
{
    AttnPlan p = {};
    p.two_heads = Hq / Hkv % 2 == 0;
    p.pairs = p.two_heads ? Hq / 2 : Hq;
    const int64_t rows = p.two_heads ? 128 : 256, sms = device_sm_count();
    // With four items an SM, longest first, the last ones leave no SM idle for long; and parts of
    // items of up to 8 steps would cost about what they save (3 steps each, and the join's launch).
    p.split = (T + rows - 1) / rows * p.pairs < 4 * sms && keys > 8 * 128;
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
