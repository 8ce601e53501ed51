// attn_simt.cu -- causal attention on the CUDA cores in fp32, for packed and paged
// keys and values of every type.
//
// One warp takes one query row of one head and goes over its keys with the running
// maximum and sum of the softmax: the simplest form, bound by the loads of each
// row's own keys.
#include <cuda_fp8.h>

#include "attn.cuh"

namespace kda {
namespace {

// e4m3 code times scale
__device__ __forceinline__ float e4m3(uint8_t c)
{
    return __uint_as_float(((uint32_t)(c & 0x80u) << 24) | ((uint32_t)(c & 0x7fu) << 20)) * 0x1p120f;
}

template <typename KV, int E> __device__ __forceinline__ void load_kv(const void *base, const float *scale, int64_t row, int d0, int D, float (&x)[E])
{
    if constexpr (sizeof(KV) == 1) {
        const float s = scale[row];
        const uint8_t *p = (const uint8_t *)base + row * D + d0;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = e4m3(p[i]) * s;
    } else {
        const KV *p = (const KV *)base + row * D + d0;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = to_f32(p[i]);
    }
}

template <typename T, typename KV, int D>
__global__ void __launch_bounds__(128) attn_simt_kernel(const AttnArgs a)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, d0 = lane * E;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), t = id / a.Hq;
    const int h = (int)(id % a.Hq), hk = h / (a.Hq / a.Hkv);
    if (t >= a.T) return;
    int64_t n, first;
    int at, len;
    if (a.m > 0) {
        n = t / a.m; first = n * a.m; at = (int)(t - first); len = a.m;
    } else {   // the last sequence that starts at or before the row
        if (t >= a.cu[a.N]) return;
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        n = lo; first = a.cu[lo]; at = (int)(t - first); len = a.cu[lo + 1] - (int)first;
    }
    if (!dbg_in(t, a.bounds.tokens, kDbgTokenRow)) return;
    int keys = at + 1;
    if (a.kv.table) {
        bool bad;
        const int total = kv_length(a.kv, n, &bad);
        if (bad && lane == 0 && a.status) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
        keys = total - len + at + 1;
    }
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = to_f32(((const T *)a.q)[(t * a.Hq + h) * D + d0 + i]) * a.scale;
        o[i] = 0.f;
    }
    for (int j = 0; j < keys; ++j) {
        float k[E], v[E];
        int64_t row = (first + j) * a.Hkv + hk;
        if (a.kv.table) {
            const int64_t g = page_of(a.kv, n, j);
            row = g < 0 ? -1 : (g * a.Hkv + hk) * a.kv.page + (j & (a.kv.page - 1));
            if (g < 0 && lane == 0 && a.status) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) k[i] = v[i] = 0.f;
        if (row >= 0) {
            load_kv<KV, E>(a.kv.table ? a.kv.k : a.k, a.kv.ks, row, d0, D, k);
            load_kv<KV, E>(a.kv.table ? a.kv.v : a.v, a.kv.vs, row, d0, D, v);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
        s = warp_sum(s);
        if (s > m) {   // (a score that is not a number goes on into l and o)
            const float f = exp2f(m - s);
            l *= f;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] *= f;
            m = s;
        }
        const float p = m == -INFINITY && s == m ? 0.f : exp2f(s - m);
        l += p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = fmaf(p, v[i], o[i]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
        ((T *)a.out)[(t * a.Hq + h) * D + d0 + i] = from_f32<T>(l == 0.f ? 0.f : o[i] / l);
    if (a.lse && lane == 0) a.lse[t * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

template <typename T, typename KV> cudaError_t launch(const AttnArgs &a)
{
    const unsigned grid = (unsigned)((a.T * a.Hq + 3) / 4);
    if (a.D == 128) attn_simt_kernel<T, KV, 128><<<grid, 128, 0, a.stream>>>(a);
    else attn_simt_kernel<T, KV, 64><<<grid, 128, 0, a.stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs &a)
{
    if (a.dtype == KDA_DTYPE_FP32) return launch<float, float>(a);
    return a.kv.table && a.kv_dtype == KDA_DTYPE_E4M3 ? launch<__nv_bfloat16, uint8_t>(a) : launch<__nv_bfloat16, __nv_bfloat16>(a);
}

KDA_DBG_TAKE(dbg_take_attn_simt)

}  // namespace kda
