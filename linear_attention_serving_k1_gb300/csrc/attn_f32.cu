// attn_f32.cu -- causal attention of prompts in fp32, packed or over a paged cache.
//
//   s_j = scale q . k_j,  m = max s_j,  l = sum 2^(s_j - m),  O = sum 2^(s_j - m) v_j     (scale times log2 e)
//
// The products run on the warp-level matrix instructions in tf32 with both operands in two
// terms (three products: about as good as fp32 sums), which has about the multiply-add rate of the
// CUDA cores at fewer instructions.  A CTA takes 64 query rows of one head, a warp
// 16 of them with scores, weights and outputs in registers; tiles of 32 keys and values are
// copied to shared memory for all four warps, two tiles ahead.  CTAs of the last blocks, which
// see the most keys, come first.
//
// Where those are few, what counts is the way of one of them through its tiles, one after
// another, and a CTA takes 16 rows instead, its four warps each 16 keys of tiles of 64, with
// running maxima, sums and outputs of their own that are joined at the end.  Tiles then serve
// 16 rows and not 64.  Measured, us, wide and narrow (CTAs of 64 rows): D = 128, 256 tokens of 2
// heads (10) 45, 21; 1024 of 8 (136) 157, 135; 768 of 16 (208) 150, 149; 4096 of 16 (1040) 1732, 2893;
// D = 64 (half the shared memory, two CTAs an SM): 256 of 2 24, 13; 2048 of 8 (264) 199, 138; 2500
// of 16 (640) 378, 351; 4096 of 16 (1040) 840, 845.
//
// What bounds it: the instructions that split keys and values into terms, again in every warp (2500 tokens,
// 16/4 heads of 128: 782 us, 33 TFLOP/s).  The wide form at D = 128 spills 80 bytes a thread, the narrow ones 12 and 20.
// The keys of a row are never cut over CTAs: one token behind 30000, 16 heads, walks 470 tiles in turn (1776 us, where the
// bytes take 18).
#include <atomic>

#include "attn_warp.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

// Warps of a CTA that share its rows, each with its own sixteen of a tile's keys.
template <int D, int ALONG> struct Shape {
    static constexpr int kRows = 64 / ALONG, kKeys = ALONG == 1 ? 32 : 64, kStages = 3;
    static constexpr int kCtas = ALONG > 1 && D == 128 ? 1 : 2;
    static constexpr uint32_t kStage = 2 * kKeys * D * 4, kSmem = kStages * kStage;
};

template <int D, int ALONG> __global__ void __launch_bounds__(kThreads, Shape<D, ALONG>::kCtas) attn_f32_kernel(const AttnArgs a)
{
    using TL = Tile<float, D>;
    using SH = Shape<D, ALONG>;
    constexpr int NT = D / 8, kRows = SH::kRows, kKeys = SH::kKeys, kStages = SH::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int sh_scan[kThreads / 32], sh_n, sh_block;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int own = ALONG == 1 ? 16 * warp : 0;      // first of this warp's rows
    const int h = blockIdx.y, hk = h / (a.Hq / a.Hkv);

    // ---- the CTA's block: the blockIdx.x-th from the end
    after_previous();
    auto blocks = [&](int n) { return n < a.N ? (a.cu[n + 1] - a.cu[n] + kRows - 1) / kRows : 0; };
    int total = 0, sum;
    for (int b = 0; b < a.N; b += kThreads) {
        block_scan_excl<int>(blocks(b + tid), sh_scan, &sum);
        total += sum;
    }
    const int want = total - 1 - (int)blockIdx.x;
    if (want < 0) return;
    int before = 0;
    for (int b = 0; b < a.N && before <= want; b += kThreads) {
        const int x = blocks(b + tid), at = before + block_scan_excl<int>(x, sh_scan, &sum);
        if (want >= at && want < at + x) {
            sh_n = b + tid;
            sh_block = want - at;
        }
        before += sum;
    }
    __syncthreads();
    const int n = sh_n, first = a.cu[n], len = a.cu[n + 1] - first, at0 = sh_block * kRows;
    bool bad;
    const int have = a.kv.table ? kv_length(a.kv, n, &bad) : len, past = have - len;
    const int keys = past + (at0 + kRows < len ? at0 + kRows : len), tiles = keys > 0 ? (keys + kKeys - 1) / kKeys : 0;

    // ---- loads: a warp a row at a time (two at D = 64)
    const uint32_t base = tc::smem_u32(smem);
    auto load = [&](int t) {
        if (t < tiles) {
            const uint32_t kd = base + (uint32_t)(t % kStages) * SH::kStage, vd = kd + kKeys * D * 4;
            constexpr int RP = 32 / TL::kPieces, PASS = 4 * RP;
            const int pc = lane % TL::kPieces;
            int64_t page[kKeys / 16] = {};
            if (a.kv.table)
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i) {
                    const int key = t * kKeys + 16 * i;
                    page[i] = key < have ? page_of(a.kv, n, key) : -1;
                    if (key < have && page[i] < 0 && a.status && tid == 0) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
                }
#pragma unroll
            for (int i = 0; i < kKeys / PASS; ++i) {
                const int r = i * PASS + warp * RP + lane / TL::kPieces, key = t * kKeys + r;
                int64_t row = key < have ? ((int64_t)first + key) * a.Hkv + hk : -1;
                if (a.kv.table) {
                    const int64_t pg = page[i * PASS / 16];
                    row = key < have && pg >= 0 ? (pg * a.Hkv + hk) * a.kv.page + (key & (a.kv.page - 1)) : -1;
                }
                const float *k = (const float *)(a.kv.table ? a.kv.k : a.k), *v = (const float *)(a.kv.table ? a.kv.v : a.v);
                const int64_t from = row < 0 ? 0 : row * D + pc * 4;
                cp16(kd + TL::k_at(r, pc), k + from, row < 0 ? 0 : 16);
                cp16(vd + TL::v_at(r, pc), v + from, row < 0 ? 0 : 16);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int t = 0; t < kStages - 1; ++t) load(t);

    const float scale = 4.f * a.scale;           // scores come as quarters, outputs as halves
    float q[NT][4], o[NT][4], mx[2], l[2];
    int limit[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = at0 + own + g + 8 * i;
        const int64_t t = (int64_t)first + r;
        const bool live = r < len && dbg_in(t, a.bounds.tokens, kDbgTokenRow);
        limit[i] = past + r;
        mx[i] = -INFINITY;
        l[i] = 0.f;
        const float *src = (const float *)a.q + (t * a.Hq + h) * D;
#pragma unroll
        for (int s = 0; s < NT; ++s) {
            const float2 w = live ? *reinterpret_cast<const float2 *>(src + (c + 4 * (s >> 1)) * 4 + 2 * (s & 1)) : make_float2(0.f, 0.f);
            q[s][i] = 0.5f * w.x;                // (see split_halves)
            q[s][2 + i] = 0.5f * w.y;
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int t = 0; t < tiles; ++t) {
        load(t + kStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncthreads();
        uint8_t *const kd = smem + (t % kStages) * SH::kStage, *const vd = kd + kKeys * D * 4;
        // values that are not finite, of keys that some rows do not see: zeros in the product
        // (0 times them would reach those rows), and NaN in the rows that see them
        uint32_t nan[2] = {0, 0};
        if ((t + 1) * kKeys - 1 > past + at0 && __syncthreads_or(TL::any_odd(vd, kKeys, tid, kThreads))) {
            for (int j = 0; j < kKeys; ++j)
                for (int i = 0; i < 2 * NT; ++i)
                    if (t * kKeys + j < have && TL::odd_value(vd, j, TL::dim(i >> 1, 2 * c + (i & 1)))) {
                        if (t * kKeys + j <= limit[0]) nan[0] |= 1u << i;
                        if (t * kKeys + j <= limit[1]) nan[1] |= 1u << i;
                    }
            __syncthreads();
            TL::clear_odd(vd, kKeys, tid, kThreads);
            __syncthreads();
        }
        // sixteen keys at a time (a warp whose rows see none of them has nothing to do)
#pragma unroll 1
        for (int b = ALONG == 1 ? 0 : warp; b < kKeys / 16; b += ALONG) {
            const int key0 = t * kKeys + 16 * b;
            if (key0 > past + at0 + own + 15) break;
            const bool mask = key0 + 15 > past + at0 + own;
            float s[2][4];
            scores_f32<D>(s, q, kd, 16 * b, g, c);
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[nt][e] *= scale;
                    if (mask && key0 + 8 * nt + 2 * c + (e & 1) > limit[e >> 1]) s[nt][e] = -INFINITY;
                    top[e >> 1] = fmaxf(top[e >> 1], s[nt][e]);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            }
            if (__any_sync(0xffffffffu, top[0] > mx[0] || top[1] > mx[1])) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float to = fmaxf(mx[i], top[i]), f = mx[i] == to ? 1.f : exp2f(mx[i] - to);
                    mx[i] = to;
                    l[i] *= f;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][2 * i] *= f;
                        o[j][2 * i + 1] *= f;
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w = s[nt][e] == -INFINITY ? 0.f : exp2f(s[nt][e] - mx[e >> 1]);
                    l[e >> 1] += w;
                    s[nt][e] = w;
                }
            weigh_f32<D>(o, s, vd, 16 * b, g, c);
        }
        if (nan[0] | nan[1])
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                if (nan[0] >> i & 1) o[i >> 1][i & 1] = __int_as_float(0x7fc00000);
                if (nan[1] >> i & 1) o[i >> 1][2 + (i & 1)] = __int_as_float(0x7fc00000);
            }
        __syncthreads();   // the stage is free
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    if constexpr (ALONG > 1) {
        // the warps' sums, joined in their order: row r, dims 4 d .. of a thread
        constexpr int W = D + 4;
        float *const sums = reinterpret_cast<float *>(smem), *const ml = sums + ALONG * 16 * W;   // (the stages are free)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = warp * 16 + g + 8 * i;
#pragma unroll
            for (int j = 0; j < NT; j += 4)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float4 *>(sums + r * W + TL::dim(j, 2 * c + e)) =
                        make_float4(o[j][2 * i + e], o[j + 1][2 * i + e], o[j + 2][2 * i + e], o[j + 3][2 * i + e]);
            if (c == 0) {
                ml[2 * r] = mx[i];
                ml[2 * r + 1] = l[i];
            }
        }
        __syncthreads();
        for (int at = tid; at < 16 * (D / 4); at += kThreads) {
            const int r = at / (D / 4), d = at % (D / 4) * 4;
            const int64_t t = (int64_t)first + at0 + r;
            if (at0 + r >= len || !dbg_in(t, a.bounds.tokens, kDbgTokenRow)) continue;
            float m = ml[2 * r], sum = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 1; w < ALONG; ++w) m = fmaxf(m, ml[2 * (16 * w + r)]);
#pragma unroll
            for (int w = 0; w < ALONG; ++w) {
                const float mw = ml[2 * (16 * w + r)], f = mw == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : exp2f(mw - m);
                const float4 y = *reinterpret_cast<const float4 *>(sums + (16 * w + r) * W + d);
                sum = fmaf(f, ml[2 * (16 * w + r) + 1], sum);
                x.x = fmaf(f, y.x, x.x);
                x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z);
                x.w = fmaf(f, y.w, x.w);
            }
            const float inv = sum == 0.f ? 0.f : 2.f / sum;
            *reinterpret_cast<float4 *>((float *)a.out + (t * a.Hq + h) * D + d) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
            if (a.lse && d == 0) a.lse[t * a.Hq + h] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718f;
        }
    }
#pragma unroll
    for (int i = 0; ALONG == 1 && i < 2; ++i) {
        const int r = at0 + own + g + 8 * i;
        const int64_t t = (int64_t)first + r;
        if (r >= len || !dbg_in(t, a.bounds.tokens, kDbgTokenRow)) continue;
        const float inv = l[i] == 0.f ? 0.f : 2.f / l[i];
        float *dst = (float *)a.out + (t * a.Hq + h) * D;
        // columns 2 c and 2 c + 1 of four accumulators are pieces 2 c and 2 c + 1 of eight
#pragma unroll
        for (int j = 0; j < NT; j += 4)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4 *>(dst + TL::dim(j, 2 * c + e)) =
                    make_float4(o[j][2 * i + e] * inv, o[j + 1][2 * i + e] * inv, o[j + 2][2 * i + e] * inv, o[j + 3][2 * i + e] * inv);
        if (a.lse && c == 0) a.lse[t * a.Hq + h] = l[i] == 0.f ? -INFINITY : (mx[i] + log2f(l[i])) * 0.69314718f;
    }
}

template <int D, int ALONG> cudaError_t launch(const AttnArgs &a, int64_t blocks)
{
    using SH = Shape<D, ALONG>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        if ((e = cudaFuncSetAttribute(attn_f32_kernel<D, ALONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SH::kSmem)) != cudaSuccess)
            return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    return launch_following(attn_f32_kernel<D, ALONG>, dim3((unsigned)blocks, (unsigned)a.Hq), kThreads, SH::kSmem, a.stream, a);
}

template <int D> cudaError_t launch(const AttnArgs &a)
{
    const int64_t ends = a.N < a.T ? a.N : a.T, wide = a.T / Shape<D, 1>::kRows + ends;
    return wide * a.Hq > (D == 128 ? 1 : 4) * (int64_t)device_sm_count() ? launch<D, 1>(a, wide) : launch<D, 4>(a, a.T / Shape<D, 4>::kRows + ends);
}

}  // namespace

cudaError_t launch_attn_f32(const AttnArgs &a) { return a.D == 128 ? launch<128>(a) : launch<64>(a); }

KDA_DBG_TAKE(dbg_take_attn_f32)

}  // namespace kda
