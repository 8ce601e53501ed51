// kv_append.cu -- rotates the new tokens' queries and keys by their positions and
// writes keys and values into the paged cache, as they are or as e4m3 with one
// power-of-two scale per token and head.
//
//   pair (a, b) of frequency f at position p:  (a cos - b sin, a sin + b cos) * rope_scale,
//   angle p f.  e4m3: s = the smallest power of two with max |x| <= 448 s, code = rn(x / s).
//
// Every element is read and written once and hardly computed with, so memory bounds
// it.  One CTA takes one token: 16 bytes a thread and row, the cosines and sines of the
// token formed once, in shared memory, for all its heads.
//
// The angle is reduced to a fraction of a turn before the sine is taken: p / (2 pi) f
// with f / (2 pi) as two floats (48 bits) and p as two exact parts, so that far positions
// keep their angle (fp32 angles are off by 0.06 at position 10^6).
//
// A power of two as the scale costs no accuracy (e4m3 has an exponent of its own), makes
// x / s exact, and code * s is a bf16 value, so that what reads the cache rounds nothing.
#include <cuda_fp8.h>

#include "attn.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float2 two_sum(float a, float b)
{
    const float s = a + b, t = s - a;
    return make_float2(s, (a - (s - t)) + (b - t));
}

// Cosine and sine of p f.  The fraction of a turn is formed as two floats, the second
// of which the sine and cosine of the first are turned by (error about that of an fp32
// rounding up to position 2^24, 2^-20 of a turn at 2^31).
__device__ __forceinline__ float2 cos_sin(int p, float f)
{
    constexpr float kHi = 0.15915494f, kLo = 6.4206382e-9f;   // 1 / (2 pi) as two floats
    const float hi = f * kHi, lo = fmaf(f, kLo, fmaf(f, kHi, -hi));
    const float big = (float)(p & ~4095), small = (float)(p & 4095);   // both exact
    const float tb = big * hi, ts = small * hi, eb = fmaf(big, hi, -tb), es = fmaf(small, hi, -ts);
    const float2 s = two_sum(tb - rintf(tb), ts - rintf(ts));
    const float rest = (eb - rintf(eb)) + (es + (s.y + (small * lo + (big * lo - rintf(big * lo)))));
    float2 r = two_sum(s.x, rest);
    r.x -= rintf(r.x);
    float si, co;
    sincospif(2.f * r.x, &si, &co);
    const float d = 6.2831853f * r.y;
    return make_float2(fmaf(-d, si, co), fmaf(d, co, si));
}

// Scale of a row whose largest magnitude is amax (which may be NaN or infinite).
__device__ __forceinline__ float row_scale(float amax)
{
    if (!(amax < __int_as_float(0x7f800000))) return __int_as_float(0x7fc00000);
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);   // biased: 2^8 x 1.75 = 448
    return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

// 16 bytes of a row: V elements.
template <typename T> struct Piece {
    static constexpr int V = 16 / (int)sizeof(T);
    static __device__ __forceinline__ void get(const uint4 &w, float (&x)[V])
    {
        const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_f32(e[i]);
    }
    static __device__ __forceinline__ void store(T *p, const float (&x)[V])
    {
        uint4 w;
        T *e = reinterpret_cast<T *>(&w);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = from_f32<T>(x[i]);
        *reinterpret_cast<uint4 *>(p) = w;
    }
};

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a)
{
    using P = Piece<T>;
    constexpr int V = P::V, L = D / V, RP = kThreads / L;   // pieces a row, rows at once
    constexpr int kAhead = 6;                               // rows of a thread that are loaded together
    __shared__ float2 cs[D / 2];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, c = tid % L, d0 = c * V;
    const int pos = a.positions[t];
    const int seq = a.table ? a.seq_ids[t] : 0;
    if (pos < 0 || seq < 0 || (a.table && seq >= a.N)) return;   // padding
    if (!dbg_in(t, a.bounds.tokens, kDbgTokenRow)) return;
    const T *q = (const T *)a.q + t * a.qs, *k = (const T *)a.k + t * a.ks, *v = (const T *)a.v + t * a.vs;
    // rows: heads of q, of k, of v (v only for the cache; whether it has a place shows below)
    const int nq = a.q_out ? a.Hq : 0, nk = a.k_out || a.table ? a.Hkv : 0, rows = nq + nk + (a.table ? a.Hkv : 0);
    auto row = [&](int r) -> const T * { return r < nq ? q + (int64_t)r * D : r < nq + nk ? k + (int64_t)(r - nq) * D : v + (int64_t)(r - nq - nk) * D; };
    const int half = a.R >> 1;
    int64_t place = -1;                          // row of head 0 in the cache, heads a page apart
    float wc[V], ws[V];                          // of this thread's elements: x cos + partner * (-+ sin)
    // (whole warps stay in the loop: rows meet in shuffles)
    for (int r0 = 0; r0 < rows; r0 += RP * kAhead) {
        uint4 raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + u * RP + tid / L;
            raw[u] = r < rows ? *reinterpret_cast<const uint4 *>(row(r) + d0) : make_uint4(0, 0, 0, 0);
        }
        if (r0 == 0) {                           // while the first rows are on their way
            if (a.table) {
                const int col = pos >> a.shift;
                const int32_t g = col < a.cols ? a.table[(int64_t)seq * a.cols + col] : -1;
                if (g >= 0 && g < a.pages) place = (int64_t)g * a.Hkv * a.page + (pos & (a.page - 1));
                else if (a.status && tid == 0) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
            }
            for (int i = tid; i < half; i += kThreads) {
                const float2 w = cos_sin(pos, a.inv_freq[i]);
                cs[i] = make_float2(w.x * a.rope_scale, w.y * a.rope_scale);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int d = d0 + i;
                const bool low = a.interleaved ? (d & 1) == 0 : d < half;
                const float2 w = d < a.R ? cs[a.interleaved ? d >> 1 : low ? d : d - half] : make_float2(1.f, 0.f);
                wc[i] = w.x;
                ws[i] = low ? -w.y : w.y;
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (r0 + u * RP >= rows) break;      // (the same for the whole CTA)
            const int r = r0 + u * RP + tid / L;
            const bool live = r < rows;
            const int kind = r < nq ? 0 : r < nq + nk ? 1 : 2, h = r - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk);
            float x[V];
            P::get(raw[u], x);
            if (half > 0) {
                // the partner of element d is d ^ 1, or d + half or d - half: then a piece of another
                // lane, or (half not a multiple of a piece) elements of two, read again
                float z[V];
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < V; ++i) z[i] = x[i ^ 1];
                } else if (half % V == 0) {
                    const int other = ((d0 < half ? d0 + half : d0 - half) / V) & (L - 1);
                    uint4 w;
                    w.x = __shfl_sync(0xffffffffu, raw[u].x, other, L);
                    w.y = __shfl_sync(0xffffffffu, raw[u].y, other, L);
                    w.z = __shfl_sync(0xffffffffu, raw[u].z, other, L);
                    w.w = __shfl_sync(0xffffffffu, raw[u].w, other, L);
                    P::get(w, z);
                } else {
                    const T *src = row(live ? r : 0);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int d = d0 + i;
                        z[i] = d < a.R ? to_f32(src[d < half ? d + half : d - half]) : 0.f;
                    }
                }
                if (kind < 2)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (d0 + i < a.R) x[i] = x[i] * wc[i] + z[i] * ws[i];
                __syncwarp();   // a row may be written where it was read
            }
            if (live && kind == 0) P::store((T *)a.q_out + (t * a.Hq + h) * D + d0, x);
            if (live && kind == 1 && a.k_out) P::store((T *)a.k_out + (t * a.Hkv + h) * D + d0, x);
            const bool cached = live && kind > 0 && place >= 0;
            const int64_t at = place + (int64_t)h * a.page;
            if (!E4M3) {
                if (cached) P::store((T *)(kind == 1 ? a.k_cache : a.v_cache) + at * D + d0, x);
            } else {
                // (fmaxf drops NaN: one is looked for apart)
                float top = 0.f;
                bool odd = false;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    top = fmaxf(top, fabsf(x[i]));
                    odd = odd || x[i] != x[i];
                }
                if (odd) top = __int_as_float(0x7f800000);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o, L));
                const float s = row_scale(top);
                // 1 / s of a power of two from 2^-126 to 2^120 is exact
                const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));
                if (cached) {
                    uint16_t w[V / 2];
#pragma unroll
                    for (int i = 0; i < V; i += 2)
                        w[i / 2] = __nv_cvt_float2_to_fp8x2(make_float2(x[i] * inv, x[i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                    uint8_t *dst = (uint8_t *)(kind == 1 ? a.k_cache : a.v_cache) + at * D + d0;
                    if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
                    else *reinterpret_cast<uint32_t *>(dst) = w[0] | (uint32_t)w[1] << 16;
                    if (c == 0) (kind == 1 ? a.k_scale : a.v_scale)[at] = s;
                }
            }
        }
    }
}

template <typename T, bool E4M3> cudaError_t launch(const AppendArgs &a)
{
    if (a.D == 128) kv_append_kernel<T, 128, E4M3><<<(unsigned)a.T, kThreads, 0, a.stream>>>(a);
    else kv_append_kernel<T, 64, E4M3><<<(unsigned)a.T, kThreads, 0, a.stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a)
{
    if (a.dtype == KDA_DTYPE_FP32) return launch<float, false>(a);
    return a.kv_dtype == KDA_DTYPE_E4M3 && a.table ? launch<__nv_bfloat16, true>(a) : launch<__nv_bfloat16, false>(a);
}

KDA_DBG_TAKE(dbg_take_kv_append)

}  // namespace kda
