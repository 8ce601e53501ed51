// gdn_scan.cu -- the gated delta rule token by token on the CUDA cores (fp32
// inputs, and short sequences of either type), and the sequence table of a
// prefill call.
//
// The columns of a state are independent, so a warp keeps 8 columns of one
// (sequence, value head) in registers for the whole sequence and needs no
// other warp: lane (rg = lane & 7, cg = lane >> 3) holds rows 4 (8 i + rg) + j
// of columns 2 cg, 2 cg + 1.  Per token it forms S^T k and S^T q from the state
// as it is (the decay is a scalar, applied to the sums), adds them over the 8
// lanes of a column pair, and updates S <- a S + k u^T: about 190 instructions
// on the chain from one token to the next, which is what bounds a call with
// few sequences.  A CTA of 4 warps (32 columns) stages blocks of 16 tokens in
// shared memory, rows already normalised, while the next block's loads are in
// flight.
#include "gdn.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- sequence table
constexpr int kTabThreads = 1024;
constexpr int kBuckets = 1024;

__device__ __forceinline__ int32_t block_scan_excl(int32_t x, int32_t *sh, int32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();   // sh is free of its previous use
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int32_t w = sh[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        sh[lane] = w;
    }
    __syncthreads();
    *total = sh[31];
    return v - x + (warp > 0 ? sh[warp - 1] : 0);
}

// Validated offsets, first checkpoint slots, and the sequences by descending
// length (a counting sort over 1024 length classes: the order inside a class
// is arbitrary and changes no result).  One CTA.
__global__ void __launch_bounds__(kTabThreads)
gdn_table_kernel(const int32_t *__restrict__ cu_in, int N, int64_t T, int stride, int64_t capacity, GdnTable tab,
                 DevStatus *st)
{
    __shared__ int32_t sh[32], bucket[kBuckets], bad, longest;
    const int tid = threadIdx.x;
    if (tid == 0) {
        bad = 0;
        longest = 0;
        *tab.next = 0;
    }
    bucket[tid] = 0;
    __syncthreads();
    const int32_t each = (int32_t)(T / N);
    auto at = [&](int n) { return cu_in ? cu_in[n] : each * n; };
    int32_t mx = 0;
    for (int n = tid; n < N; n += kTabThreads) {
        const int32_t c0 = at(n), c1 = at(n + 1);
        if (c1 < c0 || (n == 0 && c0 != 0) || (n == N - 1 && (int64_t)c1 > T)) bad = 1;
        mx = max(mx, c1 - c0);
    }
    atomicMax(&longest, mx);
    __syncthreads();
    const bool ok = bad == 0;
    const int per = max(1, (longest + kBuckets - 1) / kBuckets);   // tokens per length class
    auto cls = [&](int32_t len) { return kBuckets - 1 - min(kBuckets - 1, len / per); };
    // contiguous runs of sequences per thread
    const int run = (N + kTabThreads - 1) / kTabThreads, n0 = min(N, tid * run), n1 = min(N, n0 + run);
    int32_t ck = 0;
    for (int n = n0; n < n1; ++n) {
        const int32_t len = ok ? at(n + 1) - at(n) : 0;
        if (stride > 0) ck += len / stride;
        atomicAdd(&bucket[cls(len)], 1);
    }
    int32_t total;
    int32_t off = block_scan_excl(ck, sh, &total);
    for (int n = n0; n < n1; ++n) {
        tab.cu[n] = ok ? at(n) : 0;
        tab.ckpt_off[n] = off;
        if (stride > 0 && ok) off += (at(n + 1) - at(n)) / stride;
    }
    if (tid == 0) {
        tab.cu[N] = ok ? at(N) : 0;
        tab.ckpt_off[N] = total;
        st->code = !ok ? (int32_t)KDA_ERR_INVALID_ARG
                       : (stride > 0 && (int64_t)total > capacity) ? (int32_t)KDA_ERR_CKPT_OVERFLOW : 0;
    }
    int32_t all;
    const int32_t mine = bucket[tid];   // (every count was made before the scan's barriers)
    const int32_t first = block_scan_excl(mine, sh, &all);
    bucket[tid] = first;
    __syncthreads();
    for (int n = n0; n < n1; ++n) {
        const int32_t len = ok ? at(n + 1) - at(n) : 0;
        tab.order[atomicAdd(&bucket[cls(len)], 1)] = n;
    }
}

// ---------------------------------------------------------------- recurrence
constexpr int TB = 16;          // tokens per staged block
constexpr int kWarps = 4;
constexpr int kCols = 8 * kWarps;

template <int DK, typename T>
__global__ void __launch_bounds__(32 * kWarps)
gdn_scan_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                const float *__restrict__ g, const float *__restrict__ beta, T *__restrict__ out, int Hk, int Hv,
                int Dv, GdnTable tab, StateIO io, Bounds bd)
{
    constexpr int IR = DK / 32;        // groups of 4 rows per lane
    constexpr int EPT = DK / 4;        // elements of one q or k row per staging thread (4 threads a row)
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ __align__(16) float sq_[TB][DK], sk_[TB][DK], sv[TB][kCols], so[TB][kCols];
    __shared__ float sa[TB], sb[TB];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rg = lane & 7, cg = lane >> 3;
    const int tiles = Dv / kCols;
    const int64_t chain = blockIdx.x / tiles;
    const int col0 = (int)(blockIdx.x % tiles) * kCols;         // first column of the CTA
    const int n = tab.order[chain / Hv], h = (int)(chain % Hv), hk = h / (Hv / Hk);
    const int t0 = tab.cu[n], len0 = tab.cu[n + 1] - t0;
    const int len = dbg_rows(t0, len0, bd);
    const int64_t block = (int64_t)DK * Dv;
    const int col = col0 + 8 * warp + 2 * cg;                   // this lane's column pair

    float S[IR][4][2];
    {
        const int64_t is = io.init ? pool_slot(io.init_slots, n, io.pool) : -1;
        const bool have = is >= 0 && dbg_in(is, bd.states, kDbgState);
        const float *src = have ? io.init + (is * Hv + h) * block : nullptr;
#pragma unroll
        for (int i = 0; i < IR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = have ? *reinterpret_cast<const float2 *>(src + (int64_t)(4 * (8 * i + rg) + j) * Dv + col)
                                      : make_float2(0.f, 0.f);
                S[i][j][0] = x.x;
                S[i][j][1] = x.y;
            }
    }
    auto store = [&](float *dst) {
#pragma unroll
        for (int i = 0; i < IR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float2 *>(dst + (int64_t)(4 * (8 * i + rg) + j) * Dv + col) =
                    make_float2(S[i][j][0], S[i][j][1]);
    };

    // staging: thread (row sr of 32: 16 of q, then 16 of k; part sp of 4) loads
    // every fourth 16-byte piece of its row; the loads of a block are issued one
    // block ahead
    const int sr = tid >> 2, sp = tid & 3, st = sr & (TB - 1);
    uint4 raw[EPT / VEC];
    float pv[TB * kCols / 128], pg = 0.f;
    auto fetch = [&](int b0) {
        const bool in = b0 + st < len;
        const T *src = (sr < TB ? q : k) + ((int64_t)(t0 + b0 + st) * Hk + hk) * DK;
#pragma unroll
        for (int p = 0; p < EPT / VEC; ++p)
            raw[p] = in ? *reinterpret_cast<const uint4 *>(src + (p * 4 + sp) * VEC) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < TB * kCols / 128; ++i) {
            const int tok = (tid + 128 * i) / kCols, c = (tid + 128 * i) % kCols;
            pv[i] = b0 + tok < len ? to_f32(v[((int64_t)(t0 + b0 + tok) * Hv + h) * Dv + col0 + c]) : 0.f;
        }
        if (tid < 2 * TB) {
            const int tok = tid & (TB - 1);
            pg = b0 + tok < len ? (tid < TB ? g : beta)[(int64_t)(t0 + b0 + tok) * Hv + h] : 0.f;
        }
    };
    if (len > 0) fetch(0);

    for (int b0 = 0; b0 < len; b0 += TB) {
        __syncthreads();   // the previous block was read, its outputs written
        {
            float x[EPT], ss = 0.f;
#pragma unroll
            for (int p = 0; p < EPT / VEC; ++p) {
                const T *e = reinterpret_cast<const T *>(&raw[p]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    x[p * VEC + i] = to_f32(e[i]);
                    ss += x[p * VEC + i] * x[p * VEC + i];
                }
            }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            const float r = rsqrtf(ss + 1e-6f);
            float *dst = sr < TB ? sq_[st] : sk_[st];
#pragma unroll
            for (int p = 0; p < EPT / VEC; ++p)
#pragma unroll
                for (int i = 0; i < VEC; ++i) dst[(p * 4 + sp) * VEC + i] = x[p * VEC + i] * r;
        }
#pragma unroll
        for (int i = 0; i < TB * kCols / 128; ++i) (&sv[0][0])[tid + 128 * i] = pv[i];
        if (tid < TB) sa[tid] = expf(pg);
        else if (tid < 2 * TB) sb[tid - TB] = pg;
        __syncthreads();
        if (b0 + TB < len) fetch(b0 + TB);

        const int nt = min(TB, len - b0);
        for (int t = 0; t < nt; ++t) {
            float a0 = 0.f, a1 = 0.f, c0 = 0.f, c1 = 0.f, kq = 0.f;
            float4 kk[IR];
#pragma unroll
            for (int i = 0; i < IR; ++i) {
                kk[i] = *reinterpret_cast<const float4 *>(&sk_[t][4 * (8 * i + rg)]);
                const float4 qq = *reinterpret_cast<const float4 *>(&sq_[t][4 * (8 * i + rg)]);
                const float kf[4] = {kk[i].x, kk[i].y, kk[i].z, kk[i].w}, qf[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a0 += kf[j] * S[i][j][0];
                    a1 += kf[j] * S[i][j][1];
                    c0 += qf[j] * S[i][j][0];
                    c1 += qf[j] * S[i][j][1];
                    kq += kf[j] * qf[j];
                }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                a0 += __shfl_xor_sync(0xffffffffu, a0, o);
                a1 += __shfl_xor_sync(0xffffffffu, a1, o);
                c0 += __shfl_xor_sync(0xffffffffu, c0, o);
                c1 += __shfl_xor_sync(0xffffffffu, c1, o);
                kq += __shfl_xor_sync(0xffffffffu, kq, o);
            }
            const float a = sa[t], b = sb[t];
            const float2 vv = *reinterpret_cast<const float2 *>(&sv[t][8 * warp + 2 * cg]);
            const float u0 = b * (vv.x - a * a0), u1 = b * (vv.y - a * a1);
#pragma unroll
            for (int i = 0; i < IR; ++i) {
                const float kf[4] = {kk[i].x, kk[i].y, kk[i].z, kk[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    S[i][j][0] = a * S[i][j][0] + kf[j] * u0;
                    S[i][j][1] = a * S[i][j][1] + kf[j] * u1;
                }
            }
            if (rg == 0)
                *reinterpret_cast<float2 *>(&so[t][8 * warp + 2 * cg]) = make_float2(a * c0 + kq * u0, a * c1 + kq * u1);
            // (the stride is a multiple of 64, so a snapshot falls on a block's last token)
            if (io.stride > 0 && t == TB - 1 && (b0 + TB) % io.stride == 0 && io.ckpts) {
                const int64_t jc = (int64_t)tab.ckpt_off[n] + (b0 + TB) / io.stride - 1;
                const int64_t ps = jc < io.capacity ? pool_slot(io.ckpt_slots, jc, io.pool) : -1;
                if (ps >= 0 && dbg_in(ps, bd.ckpts, kDbgCkpt)) store(io.ckpts + (ps * Hv + h) * block);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TB * kCols / 128; ++i) {
            const int tok = (tid + 128 * i) / kCols, c = (tid + 128 * i) % kCols;
            if (tok < nt) out[((int64_t)(t0 + b0 + tok) * Hv + h) * Dv + col0 + c] = from_f32<T>(so[tok][c]);
        }
    }
    const int64_t fs = io.fin ? pool_slot(io.final_slots, n, io.pool) : -1;
    if (fs >= 0 && dbg_in(fs, bd.states, kDbgState)) store(io.fin + (fs * Hv + h) * block);
}

template <int DK, typename T> cudaError_t launch_t(const GdnArgs &a)
{
    const int64_t blocks = (int64_t)a.N * a.Hv * (a.Dv / kCols);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    gdn_scan_kernel<DK, T><<<(unsigned)blocks, 32 * kWarps, 0, a.stream>>>(
        (const T *)a.q, (const T *)a.k, (const T *)a.v, a.g, a.beta, (T *)a.out, a.Hk, a.Hv, a.Dv, a.tab, a.io,
        a.bounds);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdn_table(const GdnArgs &a)
{
    gdn_table_kernel<<<1, kTabThreads, 0, a.stream>>>(a.cu_seqlens, a.N, a.T, a.io.stride, a.io.capacity, a.tab,
                                                      a.status);
    return cudaGetLastError();
}

cudaError_t launch_gdn_scan(const GdnArgs &a)
{
    if (a.Dk == 128)
        return a.dtype == KDA_DTYPE_BF16 ? launch_t<128, __nv_bfloat16>(a) : launch_t<128, float>(a);
    return a.dtype == KDA_DTYPE_BF16 ? launch_t<64, __nv_bfloat16>(a) : launch_t<64, float>(a);
}

KDA_DBG_TAKE(dbg_take_gdn_scan)

}  // namespace kda
