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

// S += Q K^T of 16 rows and 16 keys (from row r0 of the tile at kd) in fp32: columns 2 c,
// 2 c + 1 of keys 0 .. 7 and 8 .. 15.  q: step s holds elements 2 (s & 1) + {0, 1} of the piece c + 4 (s / 2).
template <int D>
__device__ __forceinline__ void scores_f32(float (&s)[2][4], const float (&q)[D / 8][4], const uint8_t *kd, int r0, int g, int c)
{
    using TL = Tile<float, D>;
    float lo[2][4] = {};
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const uint4 w = lds16(kd + TL::k_at(r0 + 8 * nt + g, c + 4 * i));
            const float b0[2] = {__uint_as_float(w.x), __uint_as_float(w.y)}, b1[2] = {__uint_as_float(w.z), __uint_as_float(w.w)};
            tc::mma_tf32x3_apart(s[nt], lo[nt], q[2 * i], b0);
            tc::mma_tf32x3_apart(s[nt], lo[nt], q[2 * i + 1], b1);
        }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] += lo[nt][e];
}

// O += P V of those 16 keys; the first four of a step's eight keys are the even ones.
template <int D>
__device__ __forceinline__ void weigh_f32(float (&o)[D / 8][4], const float (&pr)[2][4], const uint8_t *vd, int r0, int g, int c)
{
    using TL = Tile<float, D>;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        const float a[4] = {pr[nt][0], pr[nt][2], pr[nt][1], pr[nt][3]};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 x = lds16(vd + TL::v_at(r0 + 8 * nt + 2 * c, g + 8 * i)), y = lds16(vd + TL::v_at(r0 + 8 * nt + 2 * c + 1, g + 8 * i));
            const float b[4][2] = {{__uint_as_float(x.x), __uint_as_float(y.x)}, {__uint_as_float(x.y), __uint_as_float(y.y)},
                                   {__uint_as_float(x.z), __uint_as_float(y.z)}, {__uint_as_float(x.w), __uint_as_float(y.w)}};
#pragma unroll
            for (int e = 0; e < 4; ++e) tc::mma_tf32x3(o[4 * i + e], a, b[e]);
        }
    }
}

}  // namespace kda
