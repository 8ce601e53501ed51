// gdn_scan.cu -- the gated delta rule token by token on the CUDA cores (fp32
// inputs, and short sequences of either type), and the sequence table of a
// prefill call.
//
// The columns of a state are independent, so a warp keeps 8 columns of one
// (sequence, value head) in registers for the whole sequence and needs no
// other warp: lane (rg = lane & 7, cg = lane >> 3) holds rows 4 (8 i + rg) + j
// of columns 2 cg, 2 cg + 1, as pairs of rows.  Per token it forms S^T k from the
// state as it is (the decay is a scalar, applied to the sum), adds it over the 8
// lanes of a column pair, forms S^T q meanwhile, and updates S <- a S + k u^T.
// What bounds a call is the latency of that chain from token to token (multiply-
// adds, three shuffles, the update); the next token's k is read a token ahead.
// Four more warps of the CTA stage the next 16 tokens in shared memory meanwhile,
// rows already normalised and kh . qh formed, and store the last ones' outputs.
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
        tab.next[0] = tab.next[1] = 0;
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
constexpr int kWarps = 4;       // computing warps; as many more stage
constexpr int kCols = 8 * kWarps;

template <int DK, typename T>
__global__ void __launch_bounds__(64 * kWarps)
gdn_scan_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                const float *__restrict__ g, const float *__restrict__ beta, T *__restrict__ out, int Hk, int Hv,
                int Dv, GdnTable tab, StateIO io, Bounds bd)
{
    constexpr int IR = DK / 32;        // groups of 4 rows per lane
    constexpr int EPT = DK / 4;        // elements of one q or k row per staging thread (4 threads a row)
    constexpr int VEC = 16 / (int)sizeof(T);
    // two blocks of tokens: one being computed, one being staged (and its outputs stored)
    __shared__ __align__(16) float sq_[2][TB][DK], sk_[2][TB][DK], sv[2][TB][kCols], so[2][TB][kCols];
    __shared__ float sa[2][TB], sb[2][TB], skq[2][TB];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane & 7, cg = lane >> 3;
    const bool stager = warp >= kWarps;
    const int tid = threadIdx.x & (32 * kWarps - 1);
    const int tiles = Dv / kCols;
    const int64_t chain = blockIdx.x / tiles;
    const int col0 = (int)(blockIdx.x % tiles) * kCols;         // first column of the CTA
    const int n = tab.order[chain / Hv], h = (int)(chain % Hv), hk = h / (Hv / Hk);
    const int t0 = tab.cu[n], len0 = tab.cu[n + 1] - t0;
    const int len = dbg_rows(t0, len0, bd);
    const int64_t block = (int64_t)DK * Dv;
    const int col = col0 + 8 * warp + 2 * cg;                   // a computing lane's column pair

    // Staging: thread (row sr of 32: 16 of q, then 16 of k; part sp of 4) loads
    // every fourth 16-byte piece of its row and stores it normalised.
    auto stage = [&](int b0, int buf) {
        const int sr = tid >> 2, sp = tid & 3, st = sr & (TB - 1);
        uint4 raw[EPT / VEC];
        const T *src = (sr < TB ? q : k) + ((int64_t)(t0 + b0 + st) * Hk + hk) * DK;
        const bool in = b0 + st < len;
#pragma unroll
        for (int p = 0; p < EPT / VEC; ++p)
            raw[p] = in ? *reinterpret_cast<const uint4 *>(src + (p * 4 + sp) * VEC) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < TB * kCols / 128; ++i) {
            const int tok = (tid + 128 * i) / kCols, c = (tid + 128 * i) % kCols;
            sv[buf][tok][c] = b0 + tok < len ? to_f32(v[((int64_t)(t0 + b0 + tok) * Hv + h) * Dv + col0 + c]) : 0.f;
        }
        if (tid < 2 * TB) {
            const int tok = tid & (TB - 1);
            const float x = b0 + tok < len ? (tid < TB ? g : beta)[(int64_t)(t0 + b0 + tok) * Hv + h] : 0.f;
            if (tid < TB) sa[buf][tok] = expf(x);
            else sb[buf][tok] = x;
        }
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
        float *dst = sr < TB ? sq_[buf][st] : sk_[buf][st];
#pragma unroll
        for (int p = 0; p < EPT / VEC; ++p)
#pragma unroll
            for (int i = 0; i < VEC; i += 4)
                *reinterpret_cast<float4 *>(dst + (p * 4 + sp) * VEC + i) =
                    make_float4(x[p * VEC + i] * r, x[p * VEC + i + 1] * r, x[p * VEC + i + 2] * r, x[p * VEC + i + 3] * r);
        asm volatile("bar.sync 1, 128;" ::: "memory");   // (the staging warps)
        float d = 0.f;   // kh . qh: eight threads a token
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
            const float4 y = *reinterpret_cast<const float4 *>(&sq_[buf][tid >> 3][4 * (8 * i + (tid & 7))]);
            const float4 z = *reinterpret_cast<const float4 *>(&sk_[buf][tid >> 3][4 * (8 * i + (tid & 7))]);
            d += y.x * z.x + y.y * z.y + y.z * z.z + y.w * z.w;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if ((tid & 7) == 0) skq[buf][tid >> 3] = d;
    };
    auto flush = [&](int b0, int buf) {
#pragma unroll
        for (int i = 0; i < TB * kCols / 128; ++i) {
            const int tok = (tid + 128 * i) / kCols, c = (tid + 128 * i) % kCols;
            if (b0 + tok < len) out[((int64_t)(t0 + b0 + tok) * Hv + h) * Dv + col0 + c] = from_f32<T>(so[buf][tok][c]);
        }
    };
    if (stager) {
        if (len > 0) stage(0, 0);
        __syncthreads();
        int buf = 0;
        for (int b0 = 0; b0 < len; b0 += TB, buf ^= 1) {
            // while block b0 is computed: the outputs of the one before, then the next
            if (b0 > 0) flush(b0 - TB, buf ^ 1);
            if (b0 + TB < len) stage(b0 + TB, buf ^ 1);
            __syncthreads();
        }
        if (len > 0) flush((len - 1) / TB * TB, buf ^ 1);
        return;
    }

    float2 S[IR][2][2];    // [group of 4 rows][pair of rows][column]
    {
        const int64_t is = io.init ? pool_slot(io.init_slots, n, io.pool) : -1;
        const bool have = is >= 0 && dbg_in(is, bd.states, kDbgState);
        const float *src = have ? io.init + (is * Hv + h) * block : nullptr;
#pragma unroll
        for (int i = 0; i < IR; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float *at = src + (int64_t)(4 * (8 * i + rg) + 2 * j) * Dv + col;
                const float2 x = have ? *reinterpret_cast<const float2 *>(at) : make_float2(0.f, 0.f);
                const float2 y = have ? *reinterpret_cast<const float2 *>(at + Dv) : make_float2(0.f, 0.f);
                S[i][j][0] = make_float2(x.x, y.x);
                S[i][j][1] = make_float2(x.y, y.y);
            }
    }
    auto store = [&](float *dst) {
#pragma unroll
        for (int i = 0; i < IR; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float *at = dst + (int64_t)(4 * (8 * i + rg) + 2 * j) * Dv + col;
                *reinterpret_cast<float2 *>(at) = make_float2(S[i][j][0].x, S[i][j][1].x);
                *reinterpret_cast<float2 *>(at + Dv) = make_float2(S[i][j][0].y, S[i][j][1].y);
            }
    };
    __syncthreads();
    int buf = 0;
    for (int b0 = 0; b0 < len; b0 += TB, buf ^= 1) {
        const int nt = min(TB, len - b0);
        float2 k2[IR][2];
        auto load_k = [&](int t) {
#pragma unroll
            for (int i = 0; i < IR; ++i) {
                const float4 x = *reinterpret_cast<const float4 *>(&sk_[buf][t][4 * (8 * i + rg)]);
                k2[i][0] = make_float2(x.x, x.y);
                k2[i][1] = make_float2(x.z, x.w);
            }
        };
        load_k(0);
        for (int t = 0; t < nt; ++t) {
            const float a = sa[buf][t], b = sb[buf][t], kq = skq[buf][t];
            const float2 vv = *reinterpret_cast<const float2 *>(&sv[buf][t][8 * warp + 2 * cg]);
            float2 p0[2], p1[2];   // S^T k of the two columns, even and odd pairs of rows apart
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                p0[j] = __fmul2_rn(k2[0][j], S[0][j][0]);
                p1[j] = __fmul2_rn(k2[0][j], S[0][j][1]);
#pragma unroll
                for (int i = 1; i < IR; ++i) {
                    p0[j] = __ffma2_rn(k2[i][j], S[i][j][0], p0[j]);
                    p1[j] = __ffma2_rn(k2[i][j], S[i][j][1], p1[j]);
                }
            }
            const float2 s0 = __fadd2_rn(p0[0], p0[1]), s1 = __fadd2_rn(p1[0], p1[1]);
            float a0 = s0.x + s0.y, a1 = s1.x + s1.y;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                a0 += __shfl_xor_sync(0xffffffffu, a0, o);
                a1 += __shfl_xor_sync(0xffffffffu, a1, o);
            }
            float2 q0 = make_float2(0.f, 0.f), q1 = q0;   // S^T q
#pragma unroll
            for (int i = 0; i < IR; ++i) {
                const float4 x = *reinterpret_cast<const float4 *>(&sq_[buf][t][4 * (8 * i + rg)]);
                const float2 q2[2] = {make_float2(x.x, x.y), make_float2(x.z, x.w)};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    q0 = __ffma2_rn(q2[j], S[i][j][0], q0);
                    q1 = __ffma2_rn(q2[j], S[i][j][1], q1);
                    S[i][j][0] = __fmul2_rn(make_float2(a, a), S[i][j][0]);
                    S[i][j][1] = __fmul2_rn(make_float2(a, a), S[i][j][1]);
                }
            }
            const float u0 = b * (vv.x - a * a0), u1 = b * (vv.y - a * a1);
#pragma unroll
            for (int i = 0; i < IR; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    S[i][j][0] = __ffma2_rn(k2[i][j], make_float2(u0, u0), S[i][j][0]);
                    S[i][j][1] = __ffma2_rn(k2[i][j], make_float2(u1, u1), S[i][j][1]);
                }
            if (t + 1 < nt) load_k(t + 1);
            float c0 = q0.x + q0.y, c1 = q1.x + q1.y;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                c0 += __shfl_xor_sync(0xffffffffu, c0, o);
                c1 += __shfl_xor_sync(0xffffffffu, c1, o);
            }
            if (rg == 0)
                *reinterpret_cast<float2 *>(&so[buf][t][8 * warp + 2 * cg]) = make_float2(a * c0 + kq * u0, a * c1 + kq * u1);
        }
        // (the stride is a multiple of 64, so a snapshot falls on a block's last token)
        if (io.stride > 0 && nt == TB && (b0 + TB) % io.stride == 0 && io.ckpts) {
            const int64_t jc = (int64_t)tab.ckpt_off[n] + (b0 + TB) / io.stride - 1;
            const int64_t ps = jc < io.capacity ? pool_slot(io.ckpt_slots, jc, io.pool) : -1;
            if (ps >= 0 && dbg_in(ps, bd.ckpts, kDbgCkpt)) store(io.ckpts + (ps * Hv + h) * block);
        }
        __syncthreads();
    }
    const int64_t fs = io.fin ? pool_slot(io.final_slots, n, io.pool) : -1;
    if (fs >= 0 && dbg_in(fs, bd.states, kDbgState)) store(io.fin + (fs * Hv + h) * block);
}

template <int DK, typename T> cudaError_t launch_t(const GdnArgs &a)
{
    const int64_t blocks = (int64_t)a.N * a.Hv * (a.Dv / kCols);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    gdn_scan_kernel<DK, T><<<(unsigned)blocks, 64 * kWarps, 0, a.stream>>>(
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
