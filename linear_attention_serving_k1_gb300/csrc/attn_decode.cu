// attn_decode.cu -- attention of one or a few new tokens a sequence over the paged
// cache, split over the cache's length and joined.
//
//   s_j = scale q . k_j,  m = max s_j,  l = sum 2^(s_j - m),  O = sum 2^(s_j - m) v_j     (scale times log2 e)
//   of parts of the keys: M = max m_i,  l = sum 2^(m_i - M) l_i,  O = sum 2^(m_i - M) O_i
//
// Every key and value is used by the m Hq / Hkv query rows of its head alone, so the
// cache's bytes bound the call, and what matters is that all SMs load all the time,
// whatever the lengths.  The work is the list of all (sequence, head, 64 or 128 keys); each
// CTA takes an equal share of it in that order, so a sequence is cut wherever a share
// ends.  A part that covers all keys of its rows is written out; the others go to the
// workspace, at most two a CTA, and a second kernel joins them in order of the keys.
//
// A CTA is four warps that load and compute on their own: each takes 16 of the 64 keys (e4m3: 32 of
// 128), copies them (cp.async, several tiles ahead, also across the ends of sequences) into
// shared memory of its own and keeps a running maximum, sum and output in registers; the
// warps meet only where rows end.  The products are warp-level matrix instructions with
// the query rows as the 16 rows of the tile: S = Q K^T, O += P V.  P goes in as two bf16
// terms (off by 2^-16 of itself at most, far below the output's own rounding; the matrix pipe idles).
//
// e4m3: codes become f16 (exact, one instruction for two), so the products are f16's: a row
// of q is multiplied by the power of two that brings its largest element to 1 .. 2 (others lose
// less than 2^-24 of that); a key's scale multiplies its scores; a value's scale its weights, which
// are referred to a power of two of their own for each row (unit), near the largest weight times scale
// so far, and O with them: an f16 weight is then off by at most 2^-11 of itself or 2^-25 of the
// largest.  (Codes moved to bf16 by their bits and weights in two terms took 373 us for 64 sequences
// of 4 tokens, bound by instructions.)  The elements of a row are handed to the products in an order
// in which a thread reads 16 bytes of a row at a time.
// fp32: tf32 products with both operands in two terms (attn_warp.cuh); scores come as quarters, outputs
// as halves.
#include <atomic>

#include "attn_warp.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 16;

struct Part {           // of the rows that begin in a CTA's share and end in a later one
    int64_t n;          // sequence, -1: none
    int32_t pair, slot, last, pad;   // head and row block; slot of this CTA's part; last CTA
};

struct Params {
    const void *q, *k, *v;
    const float *ks, *vs;
    void *out;
    float *lse;
    PagedKV kv;
    int N, Hq, Hkv, m, G, blocks;    // G rows of a token; blocks of 16 rows a head
    float scale;
    int32_t *status;
    float *parts;                    // [2 CTAs][16][D] outputs, then [2 CTAs][16] (m, l)
    float2 *ml;
    Part *meta;
    int64_t tokens;                  // rows the debug build lets through
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool TRANS> __device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ float2 lds_f2(const uint8_t *at) { return *reinterpret_cast<const float2 *>(at); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The two e4m3 codes in the lower half of x as f16 values (exact).
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t x)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The power of two below x >= 0 (from 2^-126 to 2^126), and one over a power of two of that range.
__device__ __forceinline__ float pow2_below(float x)
{
    const uint32_t b = __float_as_uint(x) & 0x7F800000u;
    return __uint_as_float(b < 0x00800000u ? 0x00800000u : b > 0x7E800000u ? 0x7E800000u : b);
}
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// A warp's keys and values in shared memory.
template <typename KV, int D> struct Ring : Tile<KV, D> {
    using TL = Tile<KV, D>;
    // keys of a warp at a time (32 codes are as many bytes as 16 bf16 values, and a warp's way through
    // 16 is mostly latency: 64 sequences of 4 tokens 327 us)
    static constexpr int kKeys = TL::k8 ? 32 : 16, kTile = kWarps * kKeys;
    static constexpr uint32_t kBytes = kKeys * TL::kRow;
    static constexpr uint32_t kStage = 2 * kBytes + (TL::k8 ? 8 * kKeys : 0);   // keys, values, their scales
    static constexpr int kStages = TL::k16 ? (D == 128 ? 3 : 6) : TL::k8 ? (D == 128 ? 3 : 6) : 3;
    static constexpr int kCtas = TL::k32 && D == 128 ? 1 : 2;             // an SM
    static constexpr uint32_t kSmem = kWarps * kStages * kStage;
};

// A place in the list of (sequence, head and row block, tile).
template <int TILE> struct Place {
    int64_t n, left;     // units left of the share, this one included
    int pair, tile, tiles, len;
    __device__ __forceinline__ void enter(const Params &p, int64_t seq)
    {
        bool bad;
        n = seq;
        len = kv_length(p.kv, n, &bad);
        if (bad && p.status && threadIdx.x == 0) atomicCAS(p.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
        tiles = len > TILE ? (len + TILE - 1) / TILE : 1;
    }
    __device__ __forceinline__ void next(const Params &p)
    {
        --left;
        if (++tile < tiles) return;
        tile = 0;
        if (++pair < p.Hkv * p.blocks) return;
        pair = 0;
        if (left > 0) enter(p, n + 1);
    }
};

template <typename T, typename KV, int D>
__global__ void __launch_bounds__(kThreads, Ring<KV, D>::kCtas) attn_decode_kernel(const Params p)
{
    using TL = Ring<KV, D>;
    constexpr int NT = D / 8, KN = TL::kKeys / 8, kTile = TL::kTile, kKeys = TL::kKeys;   // KN: eights of keys
    constexpr int QK = TL::k32 ? D / 8 : D / 16;     // steps of S = Q K^T
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float comb[kRows * (D + 4)];
    __shared__ float wm[kWarps][kRows], wl[kWarps][kRows];
    __shared__ int64_t sh_scan[kWarps], sh_n, sh_at;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int pairs = p.Hkv * p.blocks, rows = p.m * p.G;
    next_may_start();

    // ---- this CTA's share
    auto units = [&](int64_t n) -> int64_t {
        if (n >= p.N) return 0;
        bool bad;
        const int len = kv_length(p.kv, n, &bad);
        return (int64_t)pairs * (len > kTile ? (len + kTile - 1) / kTile : 1);
    };
    int64_t total = 0, sum;
    for (int64_t b = 0; b < p.N; b += kThreads) {
        block_scan_excl<int64_t>(units(b + tid), sh_scan, &sum);
        total += sum;
    }
    // (no more shares than units: none is empty, so the shares of a row follow each other)
    const int64_t ctas = total < gridDim.x ? total : gridDim.x, me = blockIdx.x;
    if (tid == 0) p.meta[me].n = -1;
    if (me >= ctas) return;
    const int64_t begin = total * me / ctas, end = total * (me + 1) / ctas;
    int64_t before = 0;
    for (int64_t b = 0; b < p.N && before <= begin; b += kThreads) {
        const int64_t x = units(b + tid), at = before + block_scan_excl<int64_t>(x, sh_scan, &sum);
        if (begin >= at && begin < at + x) {
            sh_n = b + tid;
            sh_at = begin - at;
        }
        before += sum;
    }
    __syncthreads();
    Place<kTile> now;
    now.left = end - begin;
    now.enter(p, sh_n);
    now.pair = (int)(sh_at / now.tiles);
    now.tile = (int)(sh_at % now.tiles);
    Place<kTile> ahead = now;

    // ---- loads
    const uint32_t mine = tc::smem_u32(smem) + (uint32_t)warp * (TL::kStages * TL::kStage);
    constexpr int HP = kKeys / 16;                   // sixteens of keys, each in one page
    int32_t page[HP];                                // -1: none (or no key there)
    auto pages_ahead = [&]() {
#pragma unroll
        for (int i = 0; i < HP; ++i) {
            const int at = ahead.tile * kTile + warp * kKeys + 16 * i;
            page[i] = -1;
            if (ahead.left <= 0 || at >= ahead.len) continue;
            page[i] = (int32_t)page_of(p.kv, ahead.n, at);
            if (page[i] < 0 && p.status && lane == 0) atomicCAS(p.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
        }
    };
    pages_ahead();
    auto load = [&](int stage) {
        if (ahead.left > 0) {
            const int at = ahead.tile * kTile + warp * kKeys;
            int64_t row0[HP];
            int valid[HP];                                              // rows of each sixteen (may be more than 16)
#pragma unroll
            for (int i = 0; i < HP; ++i) {
                valid[i] = page[i] < 0 ? 0 : ahead.len - at - 16 * i;
                row0[i] = page[i] < 0 ? 0 : ((int64_t)page[i] * p.Hkv + ahead.pair / p.blocks) * p.kv.page + ((at + 16 * i) & (p.kv.page - 1));
            }
            const uint32_t kd = mine + stage * TL::kStage, vd = kd + TL::kBytes;
            constexpr int RP = 32 / TL::kPieces;     // rows a pass of the warp
            const int r = lane / TL::kPieces, pc = lane % TL::kPieces;
#pragma unroll
            for (int which = 0; which < 2; ++which)
#pragma unroll
                for (int i = 0; i < kKeys / RP; ++i) {
                    const int hp = i * RP / 16, row = i * RP + r;
                    const uint8_t *src = (const uint8_t *)(which ? p.v : p.k) + row0[hp] * TL::kRow + (i * RP % 16) * TL::kRow + lane * 16;
                    cp16(which ? vd + TL::v_at(row, pc) : kd + TL::k_at(row, pc), src, row - 16 * hp < valid[hp] ? 16 : 0);
                }
            if (TL::k8 && lane < kKeys / 2) {
                const int i = lane % (kKeys / 4), hp = i / 4;
                const int64_t from = (HP == 1 || hp == 0 ? row0[0] : row0[HP - 1]) + 4 * (i & 3);
                const int left = 4 * ((HP == 1 || hp == 0 ? valid[0] : valid[HP - 1]) - 4 * (i & 3));
                cp16(vd + TL::kBytes + lane * 16, (lane < kKeys / 4 ? p.ks : p.vs) + from, left < 0 ? 0 : left > 16 ? 16 : left);
            }
            ahead.next(p);
            pages_ahead();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int s = 0; s < TL::kStages - 1; ++s) load(s);

    // ---- rows
    float o[NT][4], mx[2], l[2];
    float unit[2], qscale[2];                        // e4m3: see above (the scores' scale over the row's)
    int limit[2];                                    // last key that a row sees
    uint32_t qb[TL::k32 ? 1 : QK][4];
    float qf[TL::k32 ? QK : D / 8][4];
    bool fresh = true, first = true;
    int first_tile = 0;
    int stage = 0;

    while (now.left > 0) {
        const int hk = now.pair / p.blocks, block = now.pair % p.blocks;
        if (fresh) {
            fresh = false;
            first_tile = now.tile;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = block * kRows + g + 8 * i, tok = r / p.G, h = hk * p.G + r % p.G;
                const int64_t t = now.n * p.m + tok;
                const bool live = r < rows && dbg_in(t, p.tokens, kDbgTokenRow);
                limit[i] = r < rows ? now.len - p.m + tok : -1;
                const T *src = (const T *)p.q + (t * p.Hq + h) * D;
#pragma unroll
                for (int s = 0; s < QK; ++s) {
                    if constexpr (TL::k32) {
                        // dims of step s: element 2 (s & 1) + {0, 1} of the piece c + 4 (s / 2)
                        const float2 w = live ? *reinterpret_cast<const float2 *>(src + (c + 4 * (s >> 1)) * 4 + 2 * (s & 1)) : make_float2(0.f, 0.f);
                        qf[s][i] = 0.5f * w.x;
                        qf[s][2 + i] = 0.5f * w.y;
                    } else if constexpr (TL::k8) {
                        const uint2 w = live ? *reinterpret_cast<const uint2 *>(src + (c + 4 * (s >> 2)) * 16 + 4 * (s & 3)) : make_uint2(0, 0);
                        qb[s][i] = w.x;
                        qb[s][2 + i] = w.y;
                    } else {
                        qb[s][i] = live ? *reinterpret_cast<const uint32_t *>(src + s * 16 + 2 * c) : 0;
                        qb[s][2 + i] = live ? *reinterpret_cast<const uint32_t *>(src + s * 16 + 8 + 2 * c) : 0;
                    }
                }
                if constexpr (TL::k8) {
                    float big = 0.f;
#pragma unroll
                    for (int s = 0; s < QK; ++s)
#pragma unroll
                        for (int j = i; j < 4; j += 2) big = fmaxf(big, fmaxf(fabsf(bf16_lo(qb[s][j])), fabsf(bf16_hi(qb[s][j]))));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    const float to = big > 0.f ? pow2_below(big) : 1.f, by = pow2_inverse(to);
                    qscale[i] = p.scale * to;
#pragma unroll
                    for (int s = 0; s < QK; ++s)
#pragma unroll
                        for (int j = i; j < 4; j += 2) qb[s][j] = pack_f16(bf16_lo(qb[s][j]) * by, bf16_hi(qb[s][j]) * by);
                    unit[i] = 0x1p-126f;
                }
                mx[i] = -INFINITY;
                l[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(TL::kStages - 2) : "memory");
        __syncwarp();
        {
            int to = stage + TL::kStages - 1;
            load(to >= TL::kStages ? to - TL::kStages : to);   // (the stage read last time)
        }
        uint8_t *const kd = smem + warp * (TL::kStages * TL::kStage) + stage * TL::kStage, *const vd = kd + TL::kBytes;
        const uint32_t ka = mine + stage * TL::kStage, va = ka + TL::kBytes;   // the same, as the matrix loads take it
        if (++stage == TL::kStages) stage = 0;

        // ---- S = Q K^T: columns 2c, 2c + 1 of keys 0 .. 7 and 8 .. 15
        float s[KN][4] = {};
        if constexpr (TL::k16) {
#pragma unroll
            for (int i = 0; i < QK; ++i) {
                uint32_t b[4];
                ldmatrix4<false>(b, ka + TL::k_at((lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)));
                mma_bf16(s[0], qb[i], b[0], b[1]);
                mma_bf16(s[1], qb[i], b[2], b[3]);
            }
        } else if constexpr (TL::k8) {
#pragma unroll
            for (int i = 0; i < QK / 4; ++i)
#pragma unroll
                for (int nt = 0; nt < KN; ++nt) {
                    const uint4 w = lds16(kd + TL::k_at(8 * nt + g, c + 4 * i));
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16(s[nt], qb[4 * i + j], e4m3_f16x2(x[j]), e4m3_f16x2(x[j] >> 16));
                }
        } else {
            scores_f32<D>(s, qf, kd, 0, g, c);
        }

        // ---- weights
        const int key0 = now.tile * kTile + warp * kKeys;
        float ksc[KN][2], vsc[KN][2];
#pragma unroll
        for (int nt = 0; nt < KN; ++nt) {
            if constexpr (TL::k8) {
                const float2 a = lds_f2(vd + TL::kBytes + (8 * nt + 2 * c) * 4), b = lds_f2(vd + TL::kBytes + (kKeys + 8 * nt + 2 * c) * 4);
                ksc[nt][0] = a.x;
                ksc[nt][1] = a.y;
                vsc[nt][0] = b.x;
                vsc[nt][1] = b.y;
            } else {
                ksc[nt][0] = ksc[nt][1] = (TL::k32 ? 4.f : 1.f) * p.scale;
                vsc[nt][0] = vsc[nt][1] = 1.f;
            }
        }
        const bool some = key0 + kKeys - 1 > now.len - p.m;            // keys that not every row sees
#pragma unroll
        for (int nt = 0; nt < KN; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nt][e] *= TL::k8 ? ksc[nt][e & 1] * qscale[e >> 1] : ksc[nt][e & 1];
                if (some && key0 + 8 * nt + 2 * c + (e & 1) > limit[e >> 1]) s[nt][e] = -INFINITY;
            }
        float top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
            for (int nt = 1; nt < KN; ++nt) top[i] = fmaxf(top[i], fmaxf(s[nt][2 * i], s[nt][2 * i + 1]));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        }
        float fx[2] = {1.f, 1.f};
        if (__any_sync(0xffffffffu, top[0] > mx[0] || top[1] > mx[1])) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float to = fmaxf(mx[i], top[i]);
                fx[i] = mx[i] == to ? 1.f : exp2f(mx[i] - to);
                mx[i] = to;
                l[i] *= fx[i];
                if (!TL::k8)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][2 * i] *= fx[i];
                        o[j][2 * i + 1] *= fx[i];
                    }
            }
        }
        // (a masked key counts nothing, also where its value's scale is not a number)
        float pr[KN][4];
#pragma unroll
        for (int nt = 0; nt < KN; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool out = s[nt][e] == -INFINITY;
                const float w = out ? 0.f : tc::ex2_ftz(s[nt][e] - mx[e >> 1]);
                l[e >> 1] += w;
                pr[nt][e] = TL::k8 ? (out ? 0.f : w * vsc[nt][e & 1]) : w;
            }

        if constexpr (TL::k8) {
            float big[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                big[i] = fmaxf(pr[0][2 * i], pr[0][2 * i + 1]);
#pragma unroll
                for (int nt = 1; nt < KN; ++nt) big[i] = fmaxf(big[i], fmaxf(pr[nt][2 * i], pr[nt][2 * i + 1]));
                big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 1));
                big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 2));
            }
            if (__any_sync(0xffffffffu, fx[0] != 1.f || fx[1] != 1.f || big[0] > unit[0] * 16384.f || big[1] > unit[1] * 16384.f)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float was = unit[i] * fx[i], to = pow2_below(fmaxf(was, big[i])), f = was * pow2_inverse(to);
                    unit[i] = to;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[j][2 * i] *= f;
                        o[j][2 * i + 1] *= f;
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < KN; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) pr[nt][e] *= pow2_inverse(unit[e >> 1]);
        }

        // ---- values that are not finite, of keys that some rows do not see: zeros in the
        // product (0 times them would reach those rows), and NaN in the rows that see them
        uint32_t nan0 = 0, nan1 = 0;
        if constexpr (!TL::k8) {
            if (some && p.m > 1) {
                if (__any_sync(0xffffffffu, TL::any_odd(vd, kKeys, lane, 32))) {
                    for (int j = 0; j < kKeys; ++j)
                        for (int i = 0; i < 2 * NT; ++i) {
                            if (TL::odd_value(vd, j, TL::dim(i >> 1, 2 * c + (i & 1)))) {
                                if (key0 + j <= limit[0]) nan0 |= 1u << i;
                                if (key0 + j <= limit[1]) nan1 |= 1u << i;
                            }
                        }
                    __syncwarp();
                    TL::clear_odd(vd, kKeys, lane, 32);
                    __syncwarp();
                }
            }
        }

        // ---- O += P V
        if constexpr (!TL::k32) {
            uint32_t hi[KN / 2][4], lo[4];
#pragma unroll
            for (int k = 0; k < KN / 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = pr[2 * k + (i >> 1)][2 * (i & 1)], y = pr[2 * k + (i >> 1)][2 * (i & 1) + 1];
                    hi[k][i] = TL::k8 ? pack_f16(x, y) : pack_bf16(x, y);
                    if (TL::k16) lo[i] = pack_bf16(x - bf16_lo(hi[k][i]), y - bf16_hi(hi[k][i]));
                }
            if constexpr (TL::k16) {
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    uint32_t b[4];
                    ldmatrix4<true>(b, va + TL::v_at(lane & 15, 2 * j + (lane >> 4)));
                    mma_bf16(o[2 * j], hi[0], b[0], b[1]);
                    mma_bf16(o[2 * j + 1], hi[0], b[2], b[3]);
                    mma_bf16(o[2 * j], lo, b[0], b[1]);
                    mma_bf16(o[2 * j + 1], lo, b[2], b[3]);
                }
            } else {
                constexpr int W = D / 32;            // words of a thread's D / 8 codes of a row
#pragma unroll
                for (int k = 0; k < KN / 2; ++k) {
                    uint32_t x[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * k + 2 * c + (i & 1) + 8 * (i >> 1);
                        if constexpr (W == 4) {
                            const uint4 u = lds16(vd + TL::v_at(r, g));
                            x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
                        } else {
                            const float2 u = lds_f2(vd + TL::v_at(r, g >> 1) + 8 * (g & 1));
                            x[i][0] = __float_as_uint(u.x); x[i][1] = __float_as_uint(u.y);
                        }
                    }
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        // a dim of two keys side by side
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const uint32_t sel = e ? 0x7362u : 0x5140u, y0 = __byte_perm(x[0][w], x[1][w], sel), y1 = __byte_perm(x[2][w], x[3][w], sel);
                            mma_f16(o[4 * w + e], hi[k], e4m3_f16x2(y0), e4m3_f16x2(y1));
                            mma_f16(o[4 * w + e + 1], hi[k], e4m3_f16x2(y0 >> 16), e4m3_f16x2(y1 >> 16));
                        }
                }
            }
        } else {
            weigh_f32<D>(o, pr, vd, 0, g, c);
        }
        if constexpr (!TL::k8)
            if (nan0 | nan1)
#pragma unroll
                for (int i = 0; i < 2 * NT; ++i) {
                    if (nan0 >> i & 1) o[i >> 1][i & 1] = __int_as_float(0x7fc00000);
                    if (nan1 >> i & 1) o[i >> 1][2 + (i & 1)] = __int_as_float(0x7fc00000);
                }

        // ---- the rows' keys, or the share, end here
        const bool last = now.tile + 1 == now.tiles;
        if (last || now.left == 1) {
            fresh = true;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                if (c == 0) {
                    wm[warp][g + 8 * i] = mx[i];
                    wl[warp][g + 8 * i] = l[i];
                }
            }
            __syncthreads();
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float to = wm[0][g + 8 * i];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) to = fmaxf(to, wm[w][g + 8 * i]);
                f[i] = to == -INFINITY ? 0.f : exp2f(mx[i] - to);
                if (TL::k8) f[i] *= unit[i];
            }
            for (int w = 0; w < kWarps; ++w) {
                if (warp == w)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float *at = &comb[(g + 8 * (e >> 1)) * (D + 4) + TL::dim(i, 2 * c + (e & 1))];
                            const float x = o[i][e] * f[e >> 1];
                            *at = w == 0 ? x : *at + x;
                        }
                __syncthreads();
            }
            const bool whole = first_tile == 0 && last;
            const int slot = 2 * (int)me + (first ? 0 : 1);
            first = false;
            for (int r = tid / (D / 4); r < kRows; r += kThreads / (D / 4)) {
                const int row = block * kRows + r, d = tid % (D / 4) * 4;
                if (row >= rows) break;
                float to = wm[0][r], sum = 0.f;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) to = fmaxf(to, wm[w][r]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sum += to == -INFINITY ? wl[w][r] : wl[w][r] * exp2f(wm[w][r] - to);
                float4 x = *reinterpret_cast<const float4 *>(&comb[r * (D + 4) + d]);
                if (!whole) {
                    *reinterpret_cast<float4 *>(&p.parts[((int64_t)slot * kRows + r) * D + d]) = x;
                    if (d == 0) p.ml[slot * kRows + r] = make_float2(to, sum);
                    continue;
                }
                const int tok = row / p.G, h = hk * p.G + row % p.G;
                const int64_t t = now.n * p.m + tok;
                if (!dbg_in(t, p.tokens, kDbgTokenRow)) continue;
                const float inv = sum == 0.f ? 0.f : (TL::k32 ? 2.f : 1.f) / sum;
                T *dst = (T *)p.out + (t * p.Hq + h) * D + d;
                if constexpr (TL::k32)
                    *reinterpret_cast<float4 *>(dst) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
                else
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
                if (p.lse && d == 0) p.lse[t * p.Hq + h] = sum == 0.f ? -INFINITY : (to + log2f(sum)) * 0.69314718f;
            }
            if (first_tile == 0 && !last && tid == 0) {
                // the CTA whose share holds the rows' last unit
                const int64_t unit = end - 1 + (now.tiles - 1 - now.tile);
                int64_t x = (unit * ctas) / total;
                while (total * (x + 1) / ctas <= unit) ++x;
                p.meta[me] = Part{now.n, now.pair, slot, (int32_t)x, 0};
            }
            __syncthreads();   // comb, wm and wl are free
        }
        now.next(p);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Joins the parts of the rows that begin in share blockIdx.x and end in a later one: four
// rows a CTA, four groups of threads each a quarter of the parts, summed up in order.
template <typename T, int D> __global__ void __launch_bounds__(4 * D) attn_join_kernel(const Params p)
{
    constexpr int kGroups = 4, kFew = 64;
    __shared__ float2 ml[kFew][4];
    __shared__ float4 sums[kGroups][4][D / 4];
    __shared__ float ls[kGroups][4];
    after_previous();
    const Part part = p.meta[blockIdx.x];
    if (part.n < 0) return;
    const int tid = threadIdx.x, grp = tid / D, q = tid % D / (D / 4), r = blockIdx.y * 4 + q, d = tid % (D / 4) * 4;
    const int hk = part.pair / p.blocks, row = part.pair % p.blocks * kRows + r;
    const int first = blockIdx.x, count = part.last - first + 1;
    auto slot = [&](int i) { return i == 0 ? part.slot : 2 * (first + i); };
    // maxima and sums of the first parts at once (of more, from memory)
    for (int i = tid; i < 4 * min(count, kFew); i += 4 * D) ml[i / 4][i % 4] = p.ml[slot(i / 4) * kRows + blockIdx.y * 4 + i % 4];
    __syncthreads();
    auto of = [&](int i) { return i < kFew ? ml[i][q] : p.ml[slot(i) * kRows + r]; };
    const bool live = row < p.m * p.G;           // (rows that are none were not written: nothing below counts them)
    float to = -INFINITY;
    for (int i = 0; i < count; ++i) to = fmaxf(to, of(i).x);
    float sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    const int b = count * grp / kGroups, e = count * (grp + 1) / kGroups;
    if (live)
#pragma unroll 8
        for (int i = b; i < e; ++i) {
            const float2 w = of(i);
            const float4 y = *reinterpret_cast<const float4 *>(&p.parts[((int64_t)slot(i) * kRows + r) * D + d]);
            const float f = w.x == -INFINITY ? 0.f : exp2f(w.x - to);
            sum = fmaf(f, w.y, sum);
            x.x = fmaf(f, y.x, x.x);
            x.y = fmaf(f, y.y, x.y);
            x.z = fmaf(f, y.z, x.z);
            x.w = fmaf(f, y.w, x.w);
        }
    sums[grp][q][d / 4] = x;
    if (d == 0) ls[grp][q] = sum;
    __syncthreads();
    if (grp > 0 || !live) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 y = sums[i][q][d / 4];
        sum = i == 1 ? ls[0][q] + ls[1][q] : sum + ls[i][q];
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
    }
    const int tok = row / p.G, h = hk * p.G + row % p.G;
    const int64_t t = part.n * p.m + tok;
    if (!dbg_in(t, p.tokens, kDbgTokenRow)) return;
    const float inv = sum == 0.f ? 0.f : (sizeof(T) == 4 ? 2.f : 1.f) / sum;
    T *dst = (T *)p.out + (t * p.Hq + h) * D + d;
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4 *>(dst) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (p.lse && d == 0) p.lse[t * p.Hq + h] = sum == 0.f ? -INFINITY : (to + log2f(sum)) * 0.69314718f;
}

int64_t grid_of(int64_t most, int ctas)
{
    const int64_t all = device_sm_count() * ctas;
    return most < all ? most : all;
}

template <typename T, typename KV, int D> cudaError_t launch(const AttnArgs &a, Params p, int64_t most)
{
    using TL = Ring<KV, D>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        if ((e = cudaFuncSetAttribute(attn_decode_kernel<T, KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TL::kSmem)) != cudaSuccess)
            return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    const unsigned grid = (unsigned)grid_of(most, TL::kCtas);
    attn_decode_kernel<T, KV, D><<<grid, kThreads, TL::kSmem, a.stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int rows = p.m * p.G < kRows ? p.m * p.G : kRows;
    return launch_following(attn_join_kernel<T, D>, dim3(grid, (unsigned)((rows + 3) / 4)), 4 * D, 0, a.stream, p);
}

constexpr size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// At most two CTAs an SM, two parts a CTA.
size_t attn_decode_workspace(int D)
{
    const size_t ctas = 2 * (size_t)device_sm_count();
    return align256(2 * ctas * kRows * D * sizeof(float)) + align256(2 * ctas * kRows * sizeof(float2)) + align256(ctas * sizeof(Part));
}

cudaError_t launch_attn_decode(const AttnArgs &a, void *workspace)
{
    const size_t ctas = 2 * (size_t)device_sm_count();
    char *ws = (char *)workspace;
    Params p;
    p.q = a.q; p.k = a.kv.k; p.v = a.kv.v; p.ks = a.kv.ks; p.vs = a.kv.vs; p.out = a.out; p.lse = a.lse; p.kv = a.kv;
    p.N = a.N; p.Hq = a.Hq; p.Hkv = a.Hkv; p.m = a.m; p.G = a.Hq / a.Hkv; p.blocks = (a.m * p.G + kRows - 1) / kRows;
    p.scale = a.scale; p.status = a.status; p.tokens = a.bounds.tokens;
    p.parts = (float *)ws; ws += align256(2 * ctas * kRows * a.D * sizeof(float));
    p.ml = (float2 *)ws; ws += align256(2 * ctas * kRows * sizeof(float2));
    p.meta = (Part *)ws;
    // units, if every table were full
    const double most = (double)a.N * p.Hkv * p.blocks * (((int64_t)a.kv.cols * a.kv.page + 63) / 64);
    const int64_t n = most < 1e9 ? (int64_t)most : (int64_t)1e9;
    if (a.dtype == KDA_DTYPE_FP32) return a.D == 128 ? launch<float, float, 128>(a, p, n) : launch<float, float, 64>(a, p, n);
    if (a.kv_dtype == KDA_DTYPE_E4M3)
        return a.D == 128 ? launch<__nv_bfloat16, uint8_t, 128>(a, p, n) : launch<__nv_bfloat16, uint8_t, 64>(a, p, n);
    return a.D == 128 ? launch<__nv_bfloat16, __nv_bfloat16, 128>(a, p, n) : launch<__nv_bfloat16, __nv_bfloat16, 64>(a, p, n);
}

KDA_DBG_TAKE(dbg_take_attn_decode)

}  // namespace kda
