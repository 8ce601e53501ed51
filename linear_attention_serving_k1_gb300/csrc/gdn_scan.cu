// gdn_scan.cu -- the gated delta rule token by token on the CUDA cores (fp32
// inputs, and calls without a token), and the sequence table of a prefill call.
//
// The columns of a state are independent, so a warp keeps 4, 8 or 16 columns of one
// (sequence, value head) in registers for the whole sequence and needs no other warp.
// It takes four tokens at a time: with R(t, s) the decay of tokens s + 1 .. t and A_t
// that of tokens 0 .. t of the four,
//   u_t = beta_t (v_t - A_t S^T k_t) - sum over s < t of beta_t R(t, s) (k_t.k_s) u_s
//   o_t = A_t S^T q_t + sum over s <= t of R(t, s) (q_t.k_s) u_s
//   S <- A_3 S + sum of k_s R(3, s) u_s^T
// so that all eight products with S are independent of one another, their sums over
// the lanes of a column go together, and the decay costs one multiplication of S in
// four tokens (decays are factors <= 1, each the exponential of a sum of g's: none
// overflows).  What A_3's rounding leaves off is made up for by the next group's, from
// one multiple of 64 tokens to the next (where a call may resume): rounded for each
// token instead, a weak decay would be off by up to half a step times the tokens that
// the state remembers (1.1e-5 of the state at g = -0.001, 4e-7 as it is).
// A lane holds 8 rows of CW DK / 256 columns; sums over the lanes halve the values at
// each round, until a lane holds the S^T k of one column and solves it for its u.
// Four more warps of the CTA stage the next 16 tokens in shared memory meanwhile:
// rows normalised, the dot products above, loads a block ahead; and they store
// the last block's outputs.
//
// What bounds a call: with many columns the multiply-adds (a packed pair takes 2.6 to
// 3.6 cycles of a scheduler) and, next to them, shared memory's 128 bytes a cycle,
// of which each warp's copies of k and q take most; with few, the latency of a
// group of four (700 to 900 cycles).  4 x 2048 tokens, 16 heads, 128 x 128: 465 us
// (one token at a time: 558); 256 tokens, 2 heads, 64 x 64: 25 us (43).
#include "gdn.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- sequence table
constexpr int kTabThreads = 1024;
constexpr int kBuckets = 1024;

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
constexpr int kStagers = 4;     // warps that stage
// coefficients of four tokens: beta A, beta, R(3, .); beta_t R(t, s) k_t.k_s (1,0), (2,0),
// (2,1), then A_3, then (3, .); R(t, s) q_t.k_s [4][4], zero above the diagonal; A
constexpr int kCoef = 40, kKK = 12, kQK = 20, kA = 36;

// One round of a sum over lanes in which each lane goes on with one of two values:
// `keep` is what this lane keeps, `send` what the lane across `o` keeps.
__device__ __forceinline__ float halve(float keep, float send, int o)
{
    return keep + __shfl_xor_sync(0xffffffffu, send, o);
}

template <int DK, int CW, int NW>   // NW computing warps of CW columns
__global__ void __launch_bounds__(32 * (NW + kStagers), CW == 16 ? 1 : 2)
gdn_scan_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                const float *__restrict__ g, const float *__restrict__ beta, float *__restrict__ out, int Hk, int Hv,
                int Dv, GdnTable tab, StateIO io, DevStatus *status, Bounds bd)
{
    constexpr int RG = DK / 8;         // lanes that share a column, 8 rows each
    constexpr int C = CW * RG / 32;    // columns per lane
    constexpr int CL = DK / 32;        // rows of a token per lane of a staging warp
    constexpr int kCols = CW * NW;
    constexpr int EPT = DK / 4;        // elements of one q or k row per staging thread (4 threads a row)
    // two blocks of tokens: one being computed, one being staged; outputs take the place of v
    __shared__ __align__(16) float sq_[2][TB][DK], sk_[2][TB][DK], sv[2][TB][kCols];
    __shared__ __align__(16) float sg[TB], sb[TB], sa[TB / 4], coef[2][TB / 4][kCoef];   // g, beta, A_3

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rg = lane & (RG - 1), cg = lane / RG;
    const bool stager = warp >= NW;
    const int tid = threadIdx.x - 32 * NW;   // of a staging thread
    const int tiles = Dv / kCols;
    const int64_t chain = blockIdx.x / tiles;
    const int col0 = (int)(blockIdx.x % tiles) * kCols;         // first column of the CTA
    const GdnSeq seq = gdn_sequence(tab, (int)(chain / Hv), blockIdx.x == 0 && warp == 0 ? status : nullptr);
    const int n = seq.n, t0 = seq.t0, h = (int)(chain % Hv), hk = h / (Hv / Hk);
    const int len = dbg_rows(t0, seq.len, bd);
    const int64_t block = (int64_t)DK * Dv;
    const int col = col0 + CW * warp + C * cg;                  // a computing lane's first column

    // Staging: thread (row sr of 32: 16 of q, then 16 of k; part sp of 4) loads
    // every fourth 16-byte piece of its row a block ahead and stores it normalised; then
    // each staging warp forms the coefficients of four tokens.  Rows behind the sequence
    // are zero with a decay of 1: they leave the state as it is.
    // (addresses advance with the blocks; v and the outputs: NV values of one column,
    // TV tokens apart)
    constexpr int NV = TB * kCols / 128, TV = 128 / kCols;
    static_assert(NV > 0, "a value for every staging thread");
    const int sr = tid >> 2, sp = tid & 3, st = sr & (TB - 1);
    const int vc = tid % kCols, vt = tid / kCols, gt = tid & (TB - 1);
    const float *at = (sr < TB ? q : k) + ((int64_t)(t0 + st) * Hk + hk) * DK + sp * 4;
    const float *vat = v + ((int64_t)(t0 + vt) * Hv + h) * Dv + col0 + vc;
    float *oat = out + ((int64_t)(t0 + vt) * Hv + h) * Dv + col0 + vc;
    const float *gat = (tid < TB ? g : beta) + (int64_t)(t0 + gt) * Hv + h;
    const int64_t vstep = (int64_t)TV * Hv * Dv;
    float4 raw[EPT / 4];
    float vraw[NV], graw = 0.f, off = 0.f;   // off: what the group's A_3 has to make up for, relative
    auto fetch = [&](int left) {   // tokens from the block's first to the sequence's end
#pragma unroll
        for (int p = 0; p < EPT / 4; ++p)
            raw[p] = st < left ? *reinterpret_cast<const float4 *>(at + 16 * p) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) vraw[i] = vt + TV * i < left ? vat[i * vstep] : 0.f;
        if (tid < 2 * TB) graw = gt < left ? *gat : 0.f;
        at += (int64_t)TB * Hk * DK;
        vat += NV * vstep;
        gat += (int64_t)TB * Hv;
    };
    auto stage = [&](int left, int buf) {
#pragma unroll
        for (int i = 0; i < NV; ++i) sv[buf][vt + TV * i][vc] = vraw[i];
        if (tid < TB) sg[tid] = graw;
        else if (tid < 2 * TB) sb[tid - TB] = graw;
        if (tid < 32) {   // A_3 of the four groups: lane 4 j + .. forms that of group j by itself, then in order
            float x = graw;
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            // what its rounding left off, relative (where A is far below 1, its logarithm is too
            // coarse for that, and the state forgets at once)
            const bool near1 = x > -0.5f;
            const float A = expf(x), left_off = near1 ? x - log1pf(A - 1.f) : 0.f, inv = near1 ? 2.f - A : 0.f;   // (about 1 / A)
            if ((len - left) % 64 == 0) off = 0.f;
#pragma unroll
            for (int j = 0; j < TB / 4; ++j) {
                const float Aj = __shfl_sync(0xffffffffu, A, 4 * j), ij = __shfl_sync(0xffffffffu, inv, 4 * j);
                const float more = off + __shfl_sync(0xffffffffu, left_off, 4 * j), B = ij > 0.f ? fmaf(Aj, more, Aj) : Aj;
                off = ij > 0.f ? fmaf(Aj - B, ij, more) : 0.f;
                if (tid == 0) sa[j] = B;
            }
        }
        float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < EPT / 4; ++p) {
            s4.x = fmaf(raw[p].x, raw[p].x, s4.x);
            s4.y = fmaf(raw[p].y, raw[p].y, s4.y);
            s4.z = fmaf(raw[p].z, raw[p].z, s4.z);
            s4.w = fmaf(raw[p].w, raw[p].w, s4.w);
        }
        float ss = (s4.x + s4.y) + (s4.z + s4.w);
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        const float r = rsqrtf(ss + 1e-6f);
        float *dst = sr < TB ? sq_[buf][st] : sk_[buf][st];
#pragma unroll
        for (int p = 0; p < EPT / 4; ++p)
            *reinterpret_cast<float4 *>(dst + (p * 4 + sp) * 4) =
                make_float4(raw[p].x * r, raw[p].y * r, raw[p].z * r, raw[p].w * r);
        fetch(left - TB);
        asm volatile("bar.sync 1, 128;" ::: "memory");   // (the staging warps)
        // [i][j]: q_i.k_j for j <= i, k_j.k_i above the diagonal; sums over the lanes leave
        // element lane & 15 in a lane
        const int b4 = tid >> 5;
        float y[4][CL], z[4][CL], m[16];   // the lane's CL rows of the four q and k
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < CL; i += 2) {
                const float2 a2 = *reinterpret_cast<const float2 *>(&sq_[buf][4 * b4 + t][CL * lane + i]);
                const float2 b2 = *reinterpret_cast<const float2 *>(&sk_[buf][4 * b4 + t][CL * lane + i]);
                y[t][i] = a2.x; y[t][i + 1] = a2.y;
                z[t][i] = b2.x; z[t][i + 1] = b2.y;
            }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int row = e >> 2, c = e & 3;
            m[e] = 0.f;
#pragma unroll
            for (int i = 0; i < CL; ++i) m[e] = fmaf(c <= row ? y[row][i] : z[row][i], z[c][i], m[e]);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1)
#pragma unroll
            for (int e = 0; e < 8 / o; ++e) {
                const bool odd = lane & o;
                const float keep = odd ? m[2 * e + 1] : m[2 * e], send = odd ? m[2 * e] : m[2 * e + 1];
                m[e] = halve(keep, send, o);
            }
        m[0] += __shfl_xor_sync(0xffffffffu, m[0], 16);
        const float4 g4 = *reinterpret_cast<const float4 *>(&sg[4 * b4]);
        auto sum = [&](int s, int t) {     // of g over tokens s + 1 .. t; its exponential is R(t, s)
            return (s < 1 && t >= 1 ? g4.y : 0.f) + (s < 2 && t >= 2 ? g4.z : 0.f) + (s < 3 && t >= 3 ? g4.w : 0.f);
        };
        float *cf = coef[buf][b4];
        const int row = (lane >> 2) & 3, c = lane & 3;
        if (lane < 16) {
            const float f = m[0] * expf(sum(min(row, c), max(row, c)));
            cf[kQK + lane] = c <= row ? f : 0.f;
            if (c > row) cf[kKK + (c == 1 ? 0 : c == 2 ? 1 + row : 4 + row)] = f * sb[4 * b4 + c];
        } else {
            const float e = expf(row == 2 ? sum(c, 3) : g4.x + sum(0, c)), bt = sb[4 * b4 + c];   // R(3, c), or A_c
            if (row < 3) cf[4 * row + c] = row == 0 ? bt * e : row == 1 ? bt : e;
            else {
                cf[kA + c] = e;
                if (c == 3) cf[kKK + 3] = sa[b4];
            }
        }
    };
    auto flush = [&](int left, int buf) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (vt + TV * i < left) oat[i * vstep] = sv[buf][vt + TV * i][vc];
        oat += NV * vstep;
    };
    if (stager) {
        if (len > 0) {
            fetch(len);
            stage(len, 0);
        }
        __syncthreads();
        int buf = 0;
        for (int left = len; left > 0; left -= TB, buf ^= 1) {
            // while a block is computed: the outputs of the one before, then the next
            if (left < len) flush(left + TB, buf ^ 1);
            if (left > TB) stage(left - TB, buf ^ 1);
            __syncthreads();
        }
        if (len > 0) flush((len - 1) % TB + 1, buf ^ 1);
        return;
    }

    // State: pairs of rows 4 rg + 2 j, + 1 (pairs 0, 1) and RG * 4 further (2, 3); register c
    // holds column c ^ (lane & (C - 1)) of the lane's, so that sums over the lanes of a
    // column group keep register 0 everywhere
    float2 S[4][C];
    auto row_of = [&](int j) { return 4 * RG * (j >> 1) + 4 * rg + 2 * (j & 1); };
    auto turn = [&] {   // from columns in order to that order, and back
#pragma unroll
        for (int o = 1; o < C; o <<= 1)
            if (lane & o) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (!(c & o)) {
                            const float2 x = S[j][c];
                            S[j][c] = S[j][c | o];
                            S[j][c | o] = x;
                        }
            }
    };
    {
        const int64_t is = io.init ? pool_slot(io.init_slots, n, io.pool) : -1;
        const bool have = is >= 0 && dbg_in(is, bd.states, kDbgState);
        const float *src = have ? io.init + (is * Hv + h) * block : nullptr;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float *at = src + (int64_t)row_of(j) * Dv + col + c;
                S[j][c] = have ? make_float2(at[0], at[Dv]) : make_float2(0.f, 0.f);
            }
        turn();
    }
    auto store = [&](float *dst) {
        constexpr int V = C > 1 ? 2 : 1;
        turn();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < C; c += V) {
                float *at = dst + (int64_t)row_of(j) * Dv + col + c;
                if constexpr (V == 1) {
                    at[0] = S[j][c].x;
                    at[Dv] = S[j][c].y;
                } else {
                    *reinterpret_cast<float2 *>(at) = make_float2(S[j][c].x, S[j][c + 1].x);
                    *reinterpret_cast<float2 *>(at + Dv) = make_float2(S[j][c].y, S[j][c + 1].y);
                }
            }
        turn();
    };
    auto load = [&](const float *row, float2 (&x)[4]) {   // the lane's 8 values of a row
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 y = *reinterpret_cast<const float4 *>(row + 4 * (RG * i + rg));
            x[2 * i] = make_float2(y.x, y.y);
            x[2 * i + 1] = make_float2(y.z, y.w);
        }
    };
    auto dots = [&](const float2 (&x)[4], float (&d)[C]) {   // the lane's share of S^T x
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float2 y = __fmul2_rn(x[0], S[0][c]);
#pragma unroll
            for (int j = 1; j < 4; ++j) y = __ffma2_rn(x[j], S[j][c], y);
            d[c] = y.x + y.y;
        }
    };
    // the column this lane solves and writes, and its token of four for the outputs: RG / C
    // lanes share a column (with two of them, each writes a second token)
    constexpr int SH = RG / C;
    const int mine = CW * warp + C * cg + (lane & (C - 1)), tok = (lane & C ? 1 : 0) + (SH > 2 && (lane & (2 * C)) ? 2 : 0);
    __syncthreads();
    int buf = 0;
    for (int b0 = 0; b0 < len; b0 += TB, buf ^= 1) {
        const int nt = min(TB, len - b0);
        float2 kr[4][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) load(sk_[buf][s], kr[s]);
        // one round of the sums over the column's lanes, of all values at once
        auto columns = [&](float (&d)[4][C], int o) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int c = 0; c < C; c += 2 * o) d[s][c] = halve(d[s][c], d[s][c + o], o);
        };
#pragma unroll 1
        for (int t = 0; t < nt; t += 4) {
            const float *cf = coef[buf][t >> 2];
            const float4 bA = *reinterpret_cast<const float4 *>(cf), bt = *reinterpret_cast<const float4 *>(cf + 4);
            const float4 kk = *reinterpret_cast<const float4 *>(cf + kKK), k3 = *reinterpret_cast<const float4 *>(cf + kKK + 4);
            const float v0 = bt.x * sv[buf][t][mine], v1 = bt.y * sv[buf][t + 1][mine];
            const float v2 = bt.z * sv[buf][t + 2][mine], v3 = bt.w * sv[buf][t + 3][mine];
            float d[4][C], e[4][C], p[4], u[4];   // S^T k, S^T q; p: S^T k of the lane's column, u: U
#pragma unroll
            for (int s = 0; s < 4; ++s) dots(kr[s], d[s]);
#pragma unroll
            for (int o = 1; o < C; o <<= 1) columns(d, o);
#pragma unroll
            for (int s = 0; s < 4; ++s) p[s] = d[s][0] + __shfl_xor_sync(0xffffffffu, d[s][0], C);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float2 qr[4];
                load(sq_[buf][t + (s ^ tok)], qr);
                dots(qr, e[s]);
            }
#pragma unroll
            for (int o = 2; o < SH; o <<= 1)
#pragma unroll
                for (int s = 0; s < 4; ++s) p[s] += __shfl_xor_sync(0xffffffffu, p[s], o * C);
            u[0] = v0 - bA.x * p[0];
            u[1] = v1 - bA.y * p[1] - kk.x * u[0];
            u[2] = v2 - bA.z * p[2] - kk.y * u[0] - kk.z * u[1];
            u[3] = v3 - bA.w * p[3] - k3.x * u[0] - k3.y * u[1] - k3.z * u[2];
            // S <- A_3 S + sum of k_s R(3, s) u_s
            const float4 R = *reinterpret_cast<const float4 *>(cf + 8);
            const float w[4] = {R.x * u[0], R.y * u[1], R.z * u[2], u[3]};
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[j][c] = __fmul2_rn(make_float2(kk.w, kk.w), S[j][c]);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float x = c == 0 ? w[s] : __shfl_xor_sync(0xffffffffu, w[s], c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[j][c] = __ffma2_rn(kr[s][j], make_float2(x, x), S[j][c]);
                }
                if (t + 4 < nt) load(sk_[buf][t + 4 + s], kr[s]);
            }
            // o_t = A_t q_t.S + sum of R(t, s) q_t.k_s u_s, one column and token a lane; u of later
            // tokens, whose factors are zero, is left out outright: it may not be a number
            auto put = [&](float x, int at) {
                const float4 qk = *reinterpret_cast<const float4 *>(cf + kQK + 4 * at);
                const float u1 = at >= 1 ? u[1] : 0.f, u2 = at >= 2 ? u[2] : 0.f, u3 = at >= 3 ? u[3] : 0.f;
                sv[buf][t + at][mine] = cf[kA + at] * x + (qk.x * u[0] + qk.y * u1) + (qk.z * u2 + qk.w * u3);
            };
#pragma unroll
            for (int o = 1; o < C; o <<= 1) columns(e, o);
            const float x01 = halve(e[0][0], e[1][0], C), x23 = halve(e[2][0], e[3][0], C);
            __syncwarp();   // v was read
            if constexpr (SH == 2) {
                put(x01, tok);
                put(x23, tok + 2);
            } else {
                float x = halve(x01, x23, 2 * C);
                if constexpr (SH == 8) x += __shfl_xor_sync(0xffffffffu, x, 4 * C);
                if (SH < 8 || !(lane & (4 * C))) put(x, tok);
            }
        }
        // (the stride is a multiple of 64, so a snapshot falls on a block's last token)
        if (io.stride > 0 && nt == TB && (b0 + TB) % io.stride == 0 && io.ckpts) {
            const int64_t jc = (int64_t)seq.ckpt + (b0 + TB) / io.stride - 1;
            const int64_t ps = jc < io.capacity ? pool_slot(io.ckpt_slots, jc, io.pool) : -1;
            if (ps >= 0 && dbg_in(ps, bd.ckpts, kDbgCkpt)) store(io.ckpts + (ps * Hv + h) * block);
        }
        __syncthreads();
    }
    const int64_t fs = io.fin ? pool_slot(io.final_slots, n, io.pool) : -1;
    if (fs >= 0 && dbg_in(fs, bd.states, kDbgState)) store(io.fin + (fs * Hv + h) * block);
}

template <int DK, int CW, int NW> cudaError_t launch_cw(const GdnArgs &a)
{
    const int64_t blocks = (int64_t)a.N * a.Hv * (a.Dv / (CW * NW));
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    gdn_scan_kernel<DK, CW, NW><<<(unsigned)blocks, 32 * (NW + kStagers), 0, a.stream>>>(
        (const float *)a.q, (const float *)a.k, (const float *)a.v, a.g, a.beta, (float *)a.out, a.Hk, a.Hv, a.Dv, a.tab,
        a.io, a.status, a.bounds);
    return cudaGetLastError();
}

// Columns a warp, and computing warps a CTA: as few as leave every CTA an SM of its
// own, for fewer multiply-adds between a token and the next and fewer warps that share
// an SM's shared memory; a grid beyond that is bound by throughput, and 16 columns read
// each k and q least often.  512 tokens, 128 x 128 (us,
// with the table's launch of 4):
//   value heads      4      8     16     32     64    512
//   4 x 2           63     63     77    147    286   1885
//   4 x 4           69     69     68    107    203   1307
//   8 x 4           95     95     96     96    148    945
//   16 x 4         126    126    126    127    129    839
template <int DK> cudaError_t launch_dk(const GdnArgs &a)
{
    const int64_t columns = (int64_t)a.N * a.Hv * a.Dv, sms = device_sm_count();
    if (columns <= 4 * 2 * sms) return launch_cw<DK, 4, 2>(a);
    if (columns <= 4 * 4 * sms) return launch_cw<DK, 4, 4>(a);
    return columns <= 8 * 4 * sms ? launch_cw<DK, 8, 4>(a) : launch_cw<DK, 16, 4>(a);
}

}  // namespace

bool gdn_few(const GdnArgs &a)
{
    if (a.N > kGdnFew || a.segs.P > 1) return false;
    const int64_t heads = (int64_t)a.N * a.Hv, sms = device_sm_count();
    return a.dtype == KDA_DTYPE_BF16 && a.T > 0 ? heads * ((a.Dv + 127) / 128) <= sms : heads * a.Dv <= 16 * 4 * sms;
}

cudaError_t launch_gdn_table(const GdnArgs &a)
{
    gdn_table_kernel<<<1, kTabThreads, 0, a.stream>>>(a.cu_seqlens, a.N, a.T, a.io.stride, a.io.capacity, a.tab,
                                                      a.status);
    return cudaGetLastError();
}

cudaError_t launch_gdn_scan(const GdnArgs &a)
{
    return a.Dk == 128 ? launch_dk<128>(a) : launch_dk<64>(a);
}

KDA_DBG_TAKE(dbg_take_gdn_scan)

}  // namespace kda
