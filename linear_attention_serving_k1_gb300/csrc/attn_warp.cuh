// attn_warp.cuh -- what the attention kernels on the warp-level matrix instructions
// share: copies, fragments, and the place of a tile's elements in shared memory.
#pragma once

#include "attn.cuh"
#include "tc.cuh"

namespace kda {

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// (plain loads, which the compiler may move ahead of other work)
__device__ __forceinline__ uint4 lds16(const uint8_t *at) { return *reinterpret_cast<const uint4 *>(at); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Keys and values of a tile in shared memory: rows of 16-byte pieces, piece c of row r at
// place c ^ f(r), with f such that the kernels' reads meet no bank twice.
template <typename KV, int D> struct Tile {
    static constexpr int kElem = (int)sizeof(KV), kRow = D * kElem, kPieces = kRow / 16;
    static constexpr bool k8 = kElem == 1, k16 = kElem == 2, k32 = kElem == 4;
    static __device__ __forceinline__ uint32_t k_at(int r, int c)
    {
        const int f = k16 ? r & 7 : k8 && D == 64 ? 0 : (r & 1) << 2;
        return (uint32_t)(r * kRow + ((c ^ f) << 4));
    }
    static __device__ __forceinline__ uint32_t v_at(int r, int c)
    {
        const int f = k16 ? r & 7 : k8 && D == 64 ? (r >> 1) & 3 : r & 6;
        return (uint32_t)(r * kRow + ((c ^ f) << 4));
    }
    // element of a row that column 2 c + e of accumulator i holds
    static __device__ __forceinline__ int dim(int i, int c2e)
    {
        if (k16) return 8 * i + c2e;
        if (k8) return (D / 8) * c2e + i;
        return (c2e + 8 * (i >> 2)) * 4 + (i & 3);
    }
    // Whether element d of row r of the values at vd is not finite.
    static __device__ __forceinline__ bool odd_value(const uint8_t *vd, int r, int d)
    {
        const int by = d * kElem;
        const uint8_t *at = vd + v_at(r, by >> 4) + (by & 15);
        const uint32_t x = k32 ? *reinterpret_cast<const uint32_t *>(at) : (uint32_t)*reinterpret_cast<const uint16_t *>(at) << 16;
        return (x & 0x7F800000u) == 0x7F800000u;
    }
    // Whether one of the values at vd that this thread of `n` looks at is not finite; or
    // zeros in the place of those.
    static __device__ __forceinline__ bool any_odd(const uint8_t *vd, int rows, int me, int n)
    {
        bool odd = false;
        for (int i = me; i < rows * kPieces; i += n) {
            const uint4 w = lds16(vd + i * 16);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                odd = odd || (x[j] & 0x7F800000u) == 0x7F800000u || (k16 && (x[j] & 0x7F80u) == 0x7F80u);
        }
        return odd;
    }
    static __device__ __forceinline__ void clear_odd(uint8_t *vd, int rows, int me, int n)
    {
        for (int i = me; i < rows * kRow / 4; i += n) {
            uint32_t &w = *reinterpret_cast<uint32_t *>(vd + i * 4);
            uint32_t x = w;
            if ((x & 0x7F800000u) == 0x7F800000u) x = k32 ? 0u : x & 0xFFFFu;
            if (k16 && (x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
            w = x;
        }
    }
};

// fp32 products on the matrix instructions: operands in two tf32 terms, the leading one
// rounded to nearest (truncated, every product would come out too small by 2^-22 and more, all
// of them in one direction), the other one what is left.  The instructions cut off their sums'
// last bits, so a sum runs over four steps at most before it is added up in fp32: with O in the
// accumulators throughout, 4096 keys left it 3.5e-6 off, and 1e-6 so does a score of 128 elements.
struct Split {
    uint32_t hi, lo;
};
__device__ __forceinline__ Split split_f32(float x)
{
    const uint32_t h = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    return {h, __float_as_uint(x - __uint_as_float(h))};   // (a NaN stays one in the second term)
}
// Terms of halves of the four floats of w.  Those of the largest finite values themselves would be inf and -inf, and
// their products NaN, also under a weight of zero; so queries, keys and values go in halved, which changes no
// other bit down to 2^-125.  Two at a time, so that it takes no more instructions than without (64 sequences of 8192
// tokens, 16/4 heads of 128: decode 543 us, 531 without; one at a time 561, a test for values that round up to
// infinity 647).
__device__ __forceinline__ void split_halves(Split (&s)[4], const uint4 &w)
{
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 y = __fmul2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), make_float2(0.5f, 0.5f));
        const uint32_t h0 = (__float_as_uint(y.x) + 0x1000u) & 0xFFFFE000u, h1 = (__float_as_uint(y.y) + 0x1000u) & 0xFFFFE000u;
        const float2 lo = __ffma2_rn(make_float2(__uint_as_float(h0), __uint_as_float(h1)), make_float2(-1.f, -1.f), y);
        s[i] = {h0, __float_as_uint(lo.x)};
        s[i + 1] = {h1, __float_as_uint(lo.y)};
    }
}

// d += a b and lo += the products of a first and a second term.
__device__ __forceinline__ void mma_split(float (&d)[4], float (&lo)[4], const Split (&a)[4], const Split &b0, const Split &b1)
{
    const uint32_t ah[4] = {a[0].hi, a[1].hi, a[2].hi, a[3].hi}, al[4] = {a[0].lo, a[1].lo, a[2].lo, a[3].lo};
    const uint32_t bh[2] = {b0.hi, b1.hi}, bl[2] = {b0.lo, b1.lo};
    tc::mma_m16n8k8_tf32(d, ah, bh);
    tc::mma_m16n8k8_tf32(lo, al, bh);
    tc::mma_m16n8k8_tf32(lo, ah, bl);
}

// S = Q K^T / 4 of 16 rows and 16 keys (from row r0 of the tile at kd): columns 2 c, 2 c + 1 of
// keys 0 .. 7 and 8 .. 15.  q, halved: step s holds elements 2 (s & 1) + {0, 1} of the piece c + 4 (s / 2).
template <int D>
__device__ __forceinline__ void scores_f32(float (&s)[2][4], const float (&q)[D / 8][4], const uint8_t *kd, int r0, int g, int c)
{
    using TL = Tile<float, D>;
    float lo[2][4] = {};
#pragma unroll
    for (int i0 = 0; i0 < D / 16; i0 += 2) {
        float part[2][4] = {};
#pragma unroll
        for (int i = i0; i < i0 + 2; ++i) {
            Split a[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[0][e] = split_f32(q[2 * i][e]);
                a[1][e] = split_f32(q[2 * i + 1][e]);
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const uint4 w = lds16(kd + TL::k_at(r0 + 8 * nt + g, c + 4 * i));
                Split b[4];
                split_halves(b, w);
                mma_split(part[nt], lo[nt], a[0], b[0], b[1]);
                mma_split(part[nt], lo[nt], a[1], b[2], b[3]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = i0 == 0 ? part[nt][e] : s[nt][e] + part[nt][e];
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] += lo[nt][e];
}

// O += P V / 2 of 16 keys (from row r0 of the tile at vd); the first four of a step's eight keys are
// the even ones.
template <int D>
__device__ __forceinline__ void weigh_f32(float (&o)[D / 8][4], const float (&pr)[2][4], const uint8_t *vd, int r0, int g, int c)
{
    using TL = Tile<float, D>;
    Split a[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[nt][e] = split_f32(pr[nt][e >> 1 | (e & 1) << 1]);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        float d[4][4] = {}, lo[4][4] = {};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const int r = r0 + 8 * nt + 2 * c;
            const uint4 x = lds16(vd + TL::v_at(r, g + 8 * i)), y = lds16(vd + TL::v_at(r + 1, g + 8 * i));
            Split v[2][4];
            split_halves(v[0], x);
            split_halves(v[1], y);
#pragma unroll
            for (int e = 0; e < 4; ++e) mma_split(d[e], lo[e], a[nt], v[0][e], v[1][e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int f = 0; f < 4; ++f) o[4 * i + e][f] += d[e][f] + lo[e][f];
    }
}

}  // namespace kda
