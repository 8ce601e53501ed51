// gdn_decode.cu -- single-token and multi-token decode of the gated delta rule
// (one decay per token and value head, value heads sharing a query/key head),
// fp32 state updated in place.
//
//   sk = S^T kh, sq = S^T qh     one pass over the state as it was loaded; the
//                                scalar decay a = exp(g) is applied to the sums
//   u  = beta (v - a sk)
//   o  = a sq + (kh . qh) u      (= S_new^T qh, no second pass)
//   S_new = a S + kh u^T         from the same registers, one write
//
// The columns of S do not meet in any of this, so a CTA takes a tile of CT
// columns of one (sequence, value head): every element of the state is read
// and written once (8 Dk Dv bytes per head, what bounds the call), by 16-byte
// loads that are all in flight before the first of them is used.  Narrower
// tiles put more CTAs on the machine when there are few sequences; each
// repeats the token's q and k (2 Dk elements), which is why the widest tile
// that fills the machine is taken.  256 sequences of 32 heads, 128 x 128: 161 us,
// 6.65 TB/s of states (0.98 of a plain copy); one sequence 3 us.
//
// Several tokens a call: the same kernel, the tokens one after another with the state
// in registers.  There the instructions of the sums and updates bound it, next to some
// spills (five CTAs an SM leave 96 registers a thread: 40 words of 128 x 64 tiles go to
// local memory; the one-token kernel's 80 registers spill 49, behind its loads), so those
// are packed pairs of multiply-adds, and the two sums are formed by threads of their
// own (61 us for 64 sequences of four tokens; 68 without either).  Five CTAs of 64 columns
// share an SM (before the second step, 63 us: four 64, six 74, tiles of 32 columns 73;
// 128 columns 98 at first).  All products of four tokens with the state as loaded, with
// one exchange between the threads, took 77; no barrier at a token's end but two copies
// of what it guards, 65.
#include "gdn.cuh"

namespace kda {
namespace {

// MULTI: m tokens one after another with the state in registers.
template <int DK, typename T, int CT, int THREADS, bool MULTI, int MINB>
__global__ void __launch_bounds__(THREADS, MINB)
gdn_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                  const float *__restrict__ g, const float *__restrict__ beta, float *__restrict__ state,
                  T *__restrict__ out, const int32_t *__restrict__ slots, int Hk, int Hv, int Dv, int64_t pool,
                  int m_arg, const int32_t *__restrict__ commit, int32_t *status, int ahead, Bounds bd)
{
    constexpr int C4 = CT / 4;           // float4 groups per row of the tile
    constexpr int RPI = THREADS / C4;    // rows covered per pass of the CTA
    constexpr int RPT = DK / RPI;        // rows per thread
    constexpr int NW = THREADS / 32;
    static_assert(THREADS % C4 == 0 && DK % RPI == 0 && THREADS >= DK && THREADS >= 2 * CT, "shape");
    const int m = MULTI ? m_arg : 1;
    const int tiles = Dv / CT;
    const int64_t head = blockIdx.x / tiles;     // (sequence n, value head h) = n Hv + h
    const int tile = blockIdx.x % tiles;
    const int64_t n = head / Hv;
    const int h = (int)(head % Hv), hk = h / (Hv / Hk);
    const int tid = threadIdx.x, c4 = tid % C4, r0 = tid / C4;
    const int dv4 = Dv / 4;

    // slot of sequence n; one outside [0, pool) marks a padding row: no state
    // access, zero output rows
    const int64_t slot = pool_slot(slots, n, pool);
    if (slot < 0) {
        for (int t = 0; t < m; ++t)
            if (tid < CT && dbg_in(n * m + t, bd.tokens, kDbgTokenRow))
                out[((n * m + t) * Hv + h) * Dv + tile * CT + tid] = from_f32<T>(0.f);
        return;
    }
    if (!dbg_in(slot, bd.states, kDbgState)) return;
    const int ncommit = (MULTI && commit) ? min(max(commit[n], 0), m) : m;
    float4 *S = reinterpret_cast<float4 *>(state + (slot * Hv + h) * (int64_t)DK * Dv) + tile * C4;

    float2 s[RPT][2];
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const float4 x = __ldcs(S + (int64_t)(r0 + j * RPI) * dv4 + c4);
        s[j][0] = make_float2(x.x, x.y);
        s[j][1] = make_float2(x.z, x.w);
    }

    // the tile of the CTA `ahead` positions later into L2 by line prefetches
    // (whole-width tiles only: their rows are whole lines)
    if (ahead > 0 && (int64_t)blockIdx.x + ahead < gridDim.x) {
        const int64_t b2 = (int64_t)blockIdx.x + ahead, head2 = b2 / tiles;
        const int64_t sl2 = pool_slot(slots, head2 / Hv, pool);
        if (sl2 >= 0 && dbg_in(sl2, bd.states, kDbgState)) {
            const char *nx = reinterpret_cast<const char *>(state + (sl2 * Hv + head2 % Hv) * (int64_t)DK * Dv +
                                                            (b2 % tiles) * CT);
            constexpr int LPR = CT * 4 / 128;   // lines per row
            for (int i = tid; i < DK * LPR; i += THREADS)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(nx + (int64_t)(i / LPR) * Dv * 4 + (i % LPR) * 128));
        }
    }
    // repeated slots are reported by one CTA of each sequence
    if (slots && status && h == 0 && tile == 0) {
        const int32_t mine = slots[n];
        bool dup = false;
        for (int64_t i = tid; i < n; i += THREADS) dup |= slots[i] == mine;
        if (dup) atomicCAS(status, 0, (int32_t)KDA_ERR_INVALID_ARG);
    }

    __shared__ float2 sh_kq[DK];
    __shared__ __align__(16) float sh_u[CT];
    __shared__ float sh_part[3][NW];
    __shared__ __align__(16) float4 red_k[RPI][C4];
    __shared__ __align__(16) float4 red_q[RPI][C4];

    // a token's inputs, loaded one token ahead of their use
    float qn = 0.f, kn = 0.f, vn = 0.f, gn = 0.f, bn = 0.f;
    auto load = [&](int64_t row) {
        if (tid < DK) {
            qn = to_f32(q[(row * Hk + hk) * DK + tid]);
            kn = to_f32(k[(row * Hk + hk) * DK + tid]);
        }
        if (tid < CT) vn = to_f32(v[(row * Hv + h) * Dv + tile * CT + tid]);
        gn = g[row * Hv + h];
        bn = beta[row * Hv + h];
    };
    // (debug build) from a token row outside the token buffers on, the whole CTA
    // skips the tokens (a uniform condition)
    if (m > 0 && !dbg_in(n * m, bd.tokens, kDbgTokenRow)) return;
    if (m > 0) load(n * m);
    for (int t = 0; t < m; ++t) {
        const int64_t row = n * m + t;
        const float qv = qn, kv = kn, vv = vn, a = expf(gn), b = bn;
        bool more = true;
        if (MULTI && t + 1 < m) {
            more = dbg_in(row + 1, bd.tokens, kDbgTokenRow);
            if (more) load(row + 1);
        }
        const float pq = warp_sum(qv * qv), pk = warp_sum(kv * kv), pqk = warp_sum(qv * kv);
        if ((tid & 31) == 0) {
            sh_part[0][tid >> 5] = pq;
            sh_part[1][tid >> 5] = pk;
            sh_part[2][tid >> 5] = pqk;
        }
        if (tid < DK) sh_kq[tid] = make_float2(kv, qv);
        __syncthreads();
        float nq = 0.f, nk = 0.f, nqk = 0.f;
#pragma unroll
        for (int w = 0; w < DK / 32; ++w) {
            nq += sh_part[0][w];
            nk += sh_part[1][w];
            nqk += sh_part[2][w];
        }
        const float rq = rsqrtf(nq + 1e-6f), rk = rsqrtf(nk + 1e-6f);

        // S^T k and S^T q with the raw rows of q and k: the norms are scalars too
        float2 ak[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, aq[2] = {ak[0], ak[1]};
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const float2 x = sh_kq[r0 + j * RPI], kk = make_float2(x.x, x.x), qq = make_float2(x.y, x.y);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ak[i] = __ffma2_rn(kk, s[j][i], ak[i]);
                aq[i] = __ffma2_rn(qq, s[j][i], aq[i]);
            }
        }
        red_k[r0][c4] = make_float4(ak[0].x, ak[0].y, ak[1].x, ak[1].y);
        red_q[r0][c4] = make_float4(aq[0].x, aq[0].y, aq[1].x, aq[1].y);
        __syncthreads();
        // a thread per column for S^T k and u, another for S^T q and, u known, the output
        const int col = tid % CT;
        float sum = 0.f;
        if (tid < 2 * CT) {
            const float *red = reinterpret_cast<const float *>(tid < CT ? &red_k[0][0] : &red_q[0][0]);
#pragma unroll
            for (int r = 0; r < RPI; ++r) sum += red[r * CT + col];
        }
        if (tid < CT) sh_u[tid] = rk * (b * (vv - a * rk * sum));
        __syncthreads();
        if (tid >= CT && tid < 2 * CT)
            out[(row * Hv + h) * Dv + tile * CT + col] = from_f32<T>(rq * (a * sum + nqk * sh_u[col]));
        const float4 u4 = reinterpret_cast<const float4 *>(sh_u)[c4];
        const float2 u2[2] = {make_float2(u4.x, u4.y), make_float2(u4.z, u4.w)}, a2 = make_float2(a, a);
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const float x = sh_kq[r0 + j * RPI].x;
#pragma unroll
            for (int i = 0; i < 2; ++i) s[j][i] = __ffma2_rn(a2, s[j][i], __fmul2_rn(make_float2(x, x), u2[i]));
        }
        if (t + 1 == ncommit) {
#pragma unroll
            for (int j = 0; j < RPT; ++j)
                __stcs(S + (int64_t)(r0 + j * RPI) * dv4 + c4, make_float4(s[j][0].x, s[j][0].y, s[j][1].x, s[j][1].y));
        }
        if (!more) return;
        if (MULTI) __syncthreads();   // shared vectors are rewritten by the next token
    }
}

template <int DK, typename T, int CT, int THREADS, bool MULTI, int MINB>
cudaError_t launch_tile(const GdnDecodeArgs &a, int ahead)
{
    const int64_t blocks = (int64_t)a.N * a.Hv * (a.Dv / CT);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    gdn_decode_kernel<DK, T, CT, THREADS, MULTI, MINB><<<(unsigned)blocks, THREADS, 0, a.stream>>>(
        (const T *)a.q, (const T *)a.k, (const T *)a.v, a.g, a.beta, a.state, (T *)a.out, a.slots, a.Hk, a.Hv, a.Dv,
        a.pool, a.m, a.commit, a.status, ahead, a.bounds);
    return cudaGetLastError();
}

template <int DK, typename T> cudaError_t launch_t(const GdnDecodeArgs &a)
{
    const int64_t sms = device_sm_count(), heads = (int64_t)a.N * a.Hv;
    const bool wide = heads * (a.Dv / 64) >= 2 * sms;
    if (a.m > 1 || a.commit)
        return wide ? launch_tile<DK, T, 64, 128, true, 5>(a, 0) : launch_tile<DK, T, 32, 128, true, 1>(a, 0);
    if (a.Dv % 128 == 0 && heads * (a.Dv / 128) >= 2 * sms)
        return launch_tile<DK, T, 128, 256, false, 3>(a, (int)sms);
    return wide ? launch_tile<DK, T, 64, 128, false, 1>(a, 0) : launch_tile<DK, T, 32, 128, false, 1>(a, 0);
}

}  // namespace

cudaError_t launch_gdn_decode(const GdnDecodeArgs &a)
{
    if (a.Dk == 128)
        return a.dtype == KDA_DTYPE_BF16 ? launch_t<128, __nv_bfloat16>(a) : launch_t<128, float>(a);
    return a.dtype == KDA_DTYPE_BF16 ? launch_t<64, __nv_bfloat16>(a) : launch_t<64, float>(a);
}

KDA_DBG_TAKE(dbg_take_gdn_decode)

}  // namespace kda
