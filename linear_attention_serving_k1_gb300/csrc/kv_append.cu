// kv_append.cu -- rotates the new tokens' queries and keys by their positions and
// writes keys and values into the paged cache, as they are or as e4m3 with one
// power-of-two scale per token and head.
//
//   pair (a, b) of frequency f at position p:  (a cos - b sin, a sin + b cos) * rope_scale,
//   angle p f.  e4m3: s = the smallest power of two with max |x| <= 448 s, code = rn(x / s).
//
// Every element is read and written once, so memory would bound it, were the instructions about
// each 16 bytes fewer (8192 e4m3 tokens: issue slots 74 % used, 60 % of the copy rate).  One CTA takes one token: 16 bytes a thread and row, four rows of a
// thread loaded at once, the cosines and sines of the token formed once for all its heads
// while those loads are on their way.
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

// (cosine, sine) of p f times `by`, each as two floats.  The fraction of a turn is formed as
// two floats, less a whole number of quarters; both series run in fp32 behind their leading terms,
// which are kept as two floats.  Off by 2^-27 at most up to position 2^20 (against 64 bits, on
// 3 10^6 values), by that of the fraction further out (2^-20 of a turn at 2^31).
__device__ __forceinline__ void cos_sin(int p, float f, float by, float2 &first, float2 &second)
{
    constexpr float kHi = 0.15915494f, kLo = 6.4206382e-9f;   // 1 / (2 pi) as two floats
    const float hi = f * kHi, lo = fmaf(f, kLo, fmaf(f, kHi, -hi));
    const float big = (float)(p & ~4095), small = (float)(p & 4095);   // both exact
    const float tb = big * hi, ts = small * hi, eb = fmaf(big, hi, -tb), es = fmaf(small, hi, -ts);
    const float2 s = two_sum(tb - rintf(tb), ts - rintf(ts));
    const float rest = (eb - rintf(eb)) + (es + (s.y + (small * lo + (big * lo - rintf(big * lo)))));
    const float2 r = two_sum(s.x, rest);
    const float n = rintf(4.f * r.x), t = fmaf(n, -0.25f, r.x);        // exact: |t| <= 1/8
    constexpr float kTurn = 6.2831855f, kTurnLo = -1.7484556e-7f;      // 2 pi as two floats
    const float x0 = t * kTurn, x1 = fmaf(r.y, kTurn, fmaf(t, kTurnLo, fmaf(t, kTurn, -x0)));
    const float x = x0 + x1, xl = x1 - (x - x0);
    const float x2 = x * x, x2l = fmaf(2.f * x, xl, fmaf(x, x, -x2));
    // sin = x - x^3 / 6 + ..
    const float x3 = x * x2, x3l = fmaf(x, x2l, fmaf(xl, x2, fmaf(x, x2, -x3)));
    constexpr float kSixth = -1.f / 6.f, kSixthLo = (float)(-1. / 6. - (double)(-1.f / 6.f));
    const float a = kSixth * x3, al = fmaf(kSixth, x3l, fmaf(kSixthLo, x3, fmaf(kSixth, x3, -a)));
    const float more = x3 * x2 * fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 39916800.f, 1.f / 362880.f), -1.f / 5040.f), 1.f / 120.f);
    float2 si = two_sum(x, a);
    si.y += xl + (al + more);
    // cos = 1 - x^2 / 2 + ..
    float2 co = two_sum(1.f, -0.5f * x2);
    co.y += fmaf(-0.5f, x2l, x2 * x2 * fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f));
    const int quarter = (int)n;
    if (quarter & 1) {
        const float2 w = co;
        co = make_float2(-si.x, -si.y);
        si = w;
    }
    by = quarter & 2 ? -by : by;
    first = make_float2(fmaf(by, co.x, by * co.y), fmaf(by, si.x, by * si.y));
    second = make_float2(fmaf(by, co.x, -first.x) + by * co.y, fmaf(by, si.x, -first.y) + by * si.y);
}

// The larger of two magnitudes, or NaN.
__device__ __forceinline__ float max_nan(float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// Scale of a row whose largest magnitude has the bits b (of an infinity or a NaN as well).
__device__ __forceinline__ float row_scale(uint32_t b)
{
    if (b >= 0x7f800000u) return __int_as_float(0x7fc00000);
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

// (eight CTAs an SM: 64 registers, at which the e4m3 form spills 104 bytes a thread; seven CTAs, at 72 without
// spills, take 2 % longer, the bf16 form 5 %.  8192 tokens, 32/8 heads: bf16 41 us; e4m3 45.6, bound by instructions, 41 with keys turned in fp32, one row of q
// ahead 52)
template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 8) kv_append_kernel(const AppendArgs a)
{
    using P = Piece<T>;
    constexpr int V = P::V, L = D / V, RP = kThreads / L;   // pieces a row, rows at once
    constexpr int kAhead = 2;                               // rows of q of a thread that are loaded together
    // cosine and sine of pair i at slot(i), which lays what the lanes read at once side by side
    constexpr int kStep = D / 16 + 1, kSlots = 8 * kStep;
    auto slot = [](int i) { return (i & 7) * kStep + (i >> 3); };
    __shared__ float2 cs[kSlots];
    __shared__ float4 exact[E4M3 ? kSlots : 1];             // for keys: 16 bits of either, and the rest (see turn_key)
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, r0 = tid / L, c = tid % L, d0 = c * V, half = a.R >> 1;
    const int pos = a.positions[t];
    const int seq = a.table ? a.seq_ids[t] : 0;
    if (pos < 0 || seq < 0 || (a.table && seq >= a.N)) return;   // padding
    if (!dbg_in(t, a.bounds.tokens, kDbgTokenRow)) return;
    // this thread's piece of rows r0, r0 + RP, .. of q, k and v
    const T *q = (const T *)a.q + t * a.qs + r0 * D + d0, *k = (const T *)a.k + t * a.ks + r0 * D + d0, *v = (const T *)a.v + t * a.vs + r0 * D + d0;
    const int nq = a.q_out ? a.Hq : 0, nv = a.table ? a.Hkv : 0, nk = a.k_out ? a.Hkv : nv;
    auto load = [](const T *p, bool there) { return there ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0); };
    uint4 rq[kAhead], rk = load(k, r0 < nk), rv = load(v, r0 < nv);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) rq[u] = load(q + u * RP * D, r0 + u * RP < nq);

    // while those are on their way: the place in the cache (row of head 0, heads a page
    // apart), and this thread's cosines and signed sines
    int64_t place = -1;
    if (a.table) {
        const int col = pos >> a.shift;
        const int32_t g = col < a.cols ? a.table[(int64_t)seq * a.cols + col] : -1;
        if (g >= 0 && g < a.pages) place = (int64_t)g * a.Hkv * a.page + (pos & (a.page - 1));
        else if (a.status && tid == 0) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
    }
    for (int i = tid; i < half; i += kThreads) {
        float2 w, rest;
        cos_sin(pos, a.inv_freq[i], a.rope_scale, w, rest);
        cs[slot(i)] = w;
        if (E4M3) {
            const float co = __uint_as_float(__float_as_uint(w.x) & 0xFFFFFF00u), si = __uint_as_float(__float_as_uint(w.y) & 0xFFFFFF00u);
            exact[slot(i)] = make_float4(co, si, (w.x - co) + rest.x, (w.y - si) + rest.y);
        }
    }
    __syncthreads();
    const bool turned = d0 < a.R, whole = half % V == 0, low = d0 < half;
    // of the piece's elements (interleaved: of two), side by side from here on, kStep apart
    const int from = slot(a.interleaved ? d0 >> 1 : low || !turned ? d0 & (D / 2 - 1) : d0 - half);
    float wc[V], ws[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        wc[i] = 1.f;
        ws[i] = 0.f;
        if (!turned) continue;
        if (a.interleaved) {
            const float2 w = d0 + i < a.R ? cs[from + (i >> 1) * kStep] : make_float2(1.f, 0.f);
            wc[i] = w.x;
            ws[i] = i & 1 ? w.y : -w.y;
        } else if (whole) {
            const float2 w = cs[from + i * kStep];
            wc[i] = w.x;
            ws[i] = low ? -w.y : w.y;
        } else if (d0 + i < a.R) {
            const int d = d0 + i;
            const float2 w = cs[slot(d < half ? d : d - half)];
            wc[i] = w.x;
            ws[i] = d < half ? -w.y : w.y;
        }
    }
    const int other = ((low ? d0 + half : d0 - half) / V) & (L - 1);
    // the partners of the piece raw (x, of a row at src): of element d d ^ 1, or d + half or d - half: then a
    // piece of another lane, or (half not a multiple of a piece) elements of two, read again
    auto partners = [&](const uint4 &raw, const T *src, bool live, const float (&x)[V], float (&z)[V]) {
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = x[i ^ 1];
        } else if (whole) {
            uint4 w;
            w.x = __shfl_sync(0xffffffffu, raw.x, other, L);
            w.y = __shfl_sync(0xffffffffu, raw.y, other, L);
            w.z = __shfl_sync(0xffffffffu, raw.z, other, L);
            w.w = __shfl_sync(0xffffffffu, raw.w, other, L);
            P::get(w, z);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int d = d0 + i;
                z[i] = live && d < a.R ? to_f32(src[d < half ? half + i : i - half]) : 0.f;
            }
        }
    };
    // x = the piece raw of a row (at src), turned
    auto turn = [&](const uint4 &raw, const T *src, bool live, float (&x)[V]) {
        P::get(raw, x);
        if (half == 0) return;
        float z[V];
        partners(raw, src, live, x, z);
        if (turned) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (a.R % V == 0 || d0 + i < a.R) x[i] = x[i] * wc[i] + z[i] * ws[i];
        }
        __syncwarp();   // a row may be written where it was read
    };
    // The same for a key that becomes e4m3: x cos + z sin rounded to odd (towards zero, the last bit
    // set unless that is exact), so that the code is the one nearest to the sum itself and
    // not to an fp32 rounding of it, which now and then lands on the middle between two codes (of 8
    // million codes, 10).  x and z have 8 bits; of cosine and sine, 16 go into exact products, the rest
    // into a correction with what the sum of the two leaves.
    auto turn_key = [&](const uint4 &raw, const T *src, bool live, float (&x)[V]) {
        P::get(raw, x);
        if (half == 0) return;
        float z[V];
        partners(raw, src, live, x, z);
        auto minus = [](float2 p, float2 q) { return __ffma2_rn(q, make_float2(-1.f, -1.f), p); };
        // elements i and i + 1, of cosines and sines w0 and w1
        auto two = [&](int i, float z0, float z1, const float4 &w0, const float4 &w1) {
            const float2 X = make_float2(x[i], x[i + 1]), Z = make_float2(z0, z1);
            const float2 u = __fmul2_rn(X, make_float2(w0.x, w1.x)), t = __fmul2_rn(Z, make_float2(w0.y, w1.y));
            const float2 y = __fadd2_rn(u, t), b = minus(y, u), e = __fadd2_rn(minus(u, minus(y, b)), minus(t, b));
            const float2 rest = __ffma2_rn(X, make_float2(w0.z, w1.z), __ffma2_rn(Z, make_float2(w0.w, w1.w), e));
            // (an infinity stays one: its rest is not a number)
            const float inf = __int_as_float(0x7f800000);
            const bool fine0 = fabsf(y.x) < inf, fine1 = fabsf(y.y) < inf;
            x[i] = fine0 ? __fadd_rz(y.x, rest.x) : y.x;
            x[i + 1] = fine1 ? __fadd_rz(y.y, rest.y) : y.y;
            if (fine0 && rest.x != 0.f) x[i] = __uint_as_float(__float_as_uint(x[i]) | 1u);
            if (fine1 && rest.y != 0.f) x[i + 1] = __uint_as_float(__float_as_uint(x[i + 1]) | 1u);
        };
        if (turned && a.interleaved) {
#pragma unroll
            for (int i = 0; i < V; i += 2)
                if (a.R % V == 0 || d0 + i < a.R) {
                    const float4 w = exact[from + (i >> 1) * kStep];
                    two(i, -z[i], z[i + 1], w, w);
                }
        } else if (turned && whole) {
            const uint32_t flip = low ? 0x80000000u : 0u;
#pragma unroll
            for (int i = 0; i < V; i += 2)
                two(i, __uint_as_float(__float_as_uint(z[i]) ^ flip), __uint_as_float(__float_as_uint(z[i + 1]) ^ flip),
                    exact[from + i * kStep], exact[from + (i + 1) * kStep]);
        } else if (turned) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const int d = d0 + i;
                if (d >= a.R) continue;                      // (R is even)
                two(i, d < half ? -z[i] : z[i], d + 1 < half ? -z[i + 1] : z[i + 1], exact[slot(d < half ? d : d - half)],
                    exact[slot(d + 1 < half ? d + 1 : d + 1 - half)]);
            }
        }
        __syncwarp();
    };
    // a row into the cache
    auto keep = [&](const float (&x)[V], int h, bool live, void *cache, float *scale) {
        const bool cached = live && place >= 0;
        const int64_t at = place + (int64_t)h * a.page;
        if (!E4M3) {
            if (cached) P::store((T *)cache + at * D + d0, x);
            return;
        }
        float top = fabsf(x[0]);
#pragma unroll
        for (int i = 1; i < V; ++i) top = max_nan(top, fabsf(x[i]));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o, L));
        const float s = row_scale(__float_as_uint(top));
        // 1 / s of a power of two from 2^-126 to 2^120 is exact
        const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));
        if (!cached) return;
        uint16_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V; i += 2)
            w[i / 2] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
        uint8_t *dst = (uint8_t *)cache + at * D + d0;
        // (a row that holds no number says so in its scale alone: the NaN code of a value would be one under a
        // weight of zero too, in rows that do not see it)
        const uint32_t all = s == s ? ~0u : 0u;
        if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2((w[0] | (uint32_t)w[1] << 16) & all, (w[2] | (uint32_t)w[3] << 16) & all);
        else *reinterpret_cast<uint32_t *>(dst) = (w[0] | (uint32_t)w[1] << 16) & all;
        if (c == 0) scale[at] = s;
    };
    // (whole warps stay in the loops: rows meet in shuffles)
    T *qo = (T *)a.q_out + t * a.Hq * D + r0 * D + d0;
    for (int h = 0; h < nq; h += RP * kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int off = h + u * RP;
            if (off >= nq) break;                // (the same for the whole CTA)
            const bool live = r0 + off < nq;
            float x[V];
            turn(rq[u], q + (int64_t)off * D, live, x);
            if (live) P::store(qo + (int64_t)off * D, x);
            const int more = off + RP * kAhead;
            if (more < nq) rq[u] = load(q + (int64_t)more * D, r0 + more < nq);
        }
    }
    T *ko = (T *)a.k_out + t * a.Hkv * D + r0 * D + d0;
    for (int h = 0; h < nk; h += RP) {
        const bool live = r0 + h < nk;
        if (h > 0) rk = load(k + (int64_t)h * D, live);
        float x[V];
        if (E4M3) turn_key(rk, k + (int64_t)h * D, live, x);
        else turn(rk, k + (int64_t)h * D, live, x);
        if (live && a.k_out) P::store(ko + (int64_t)h * D, x);
        keep(x, r0 + h, live, a.k_cache, a.k_scale);
    }
    for (int h = 0; h < nv; h += RP) {
        const bool live = r0 + h < nv;
        if (h > 0) rv = load(v + (int64_t)h * D, live);
        float x[V];
        P::get(rv, x);
        keep(x, r0 + h, live, a.v_cache, a.v_scale);
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
