// gdn_tc.cu -- chunked prefill of the gated delta rule on the sm_103a tensor
// cores (tcgen05, accumulators and the state operands in TMEM): bf16 q, k, v,
// one decay per token and value head, fp32 state, chunks of 64 tokens.
//
// Per chunk (rows i, j < 64; b the running sum of g; rq, rk the inverse norms
// of the raw rows of Q and K):
//   G = [K; Q] K^T
//   A = strict-lower(beta_i rk_i rk_j e^(b_i - b_j) G_kk),  T = (I + A)^-1
//   P = lower(rq_i rk_j e^(b_i - b_j) G_qk)
//   X = K S,  U = T diag(beta) V - T diag(beta e^b rk) X
//   O = e^b rq (Q S) + P U
//   S <- e^(b_C) S + K^T (rk e^(b_C - b) U)
// Decays enter as differences b_i - b_j <= 0 only, kept in two floats, so no
// chunk decays too much.  The norms are scalars beside exact bf16 rows: K, Q
// and V are multiplied as they were loaded, unrounded.
//
// One CTA runs one chain (sequence, value head, tile of 128 value columns) at a
// time, all roles in one kernel, so that nothing but q, k, v, out, the gates
// and the states touches memory:
//   producer warp   TMA loads of K and Q (three stages) and V (one) chunks; takes
//                   chains off a common counter, longest sequences first
//   issuer warps (3)   the tcgen05.mma: G, and the running decays a chunk ahead of
//                   it; T V; and the chain's products
//   gate warps (4)  norms, A (fp32) and P (two bf16 terms) from G in TMEM
//   inverse warps (4)  T from A
//   chain warps (16)   the state in fp32 registers (thread: one value column, a
//                   quarter of the key rows) and the chain S -> X -> U -> S; while its
//                   products run, T as two bf16 terms
//   output warps (4)  O from Q S and P U
// The chain is transposed, (.)^T with the 128 value columns as M: its operands
// S^T, X^T, U^T are written by the threads to TMEM (A operands) and K, Q, T, P
// are B operands in shared memory as they lie: K is K-major for X and MN-major
// for the state update, from the same tile, and V is the MN-major A operand of
// T V, so that no thread reads K, Q or V but for the norms.
//
// Precision: sums are fp32.  The state's operands S, X, U and T are carried as two
// bf16 terms (hi + lo, 2^-17) against exact K and V, and T X keeps the three
// products that matter: a state comes out 4e-6 of its norm from the exact one
// (a third term, 1e-6, costs a quarter of the time again).  The outputs are made
// alike: both terms of S in Q S, and P as two terms with three products in P U, so
// that their rounding to bf16 is all that shows.
//
// Values that are not finite: the products are masked by zeros, which such a value
// would pass, to tokens before its own.  So it is replaced by zero where it comes in
// (key rows by the gate warps, gates by the G warp, values by the T V warp, which
// sums up 0 x over each tile: 160 instructions a chunk), and from its token on the
// outputs, and behind its chunk the state, become NaN: through their factors e^b rq
// and e^bC, and for a value, in its column, as they are stored, to the chain's end.
//
// What bounds it: neither memory nor the tensor cores (a fifth of the one's and a
// third of the other's time) but the chain from chunk to chunk, about 7600 cycles
// for 64 tokens: four products one after another (some 600 cycles each with their
// waits) and between them the 16 chain warps' conversions between fp32 and two
// bf16 terms, while the other roles, which fill the same schedulers, work two
// chunks ahead.  One prompt of 8192 tokens, 32 heads of 128 x 128: 366 us, in segments;
// 16 x 2048 tokens: 526 us (503 with one term of S and P in the outputs and without
// what keeps values that are not finite from earlier tokens).  Before that (the
// latter): outputs on the chain's warps 531, the inverse of alternate chunks by two
// groups of warps 563.  All roles' loops together are as large as a scheduler's
// instruction cache: a smaller loop may be faster than an unrolled one of another
// role, and where the rare code lies shows (2 to 4 % either way).
#include <cuda.h>

#include <atomic>

#include "gdn.cuh"
#include "tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kC = kGdnChunk;
constexpr int kStages = 3;
constexpr int kWorks = 4;      // ring of chains handed from the producer to the other warps
constexpr int kPRing = 3;      // chunks whose P is waiting for its products
constexpr int kGRing = kPRing + 3;
constexpr int kVRing = 4;      // chunks whose columns with a value that is not finite are kept

// warps by role; TMEM lanes 32 (w & 3) .. + 31 belong to warp w
constexpr int kChainWarps = 16, kGateWarp0 = 16, kInvWarp0 = 20, kOutWarp0 = 24, kProducerWarp = 28, kIssuerWarp = 29,
              kGramWarp = 30, kValueWarp = 31;
constexpr int kThreads = 32 * 32;
constexpr int kWorkReaders = kChainWarps + 4 + 8 + 3;   // warps that read the work ring

// registers: each SM sub-partition (16384 registers) holds eight warps, four chain
// warps, one gate, one inverse, one output warp and one of the last four,
// launched with 64 registers a thread; they are dealt out anew within that
// total, 8 x 64 = 4 x 72 + 4 x 56.  With fewer, values spill to local memory, for
// which this kernel's shared memory leaves almost no cache: a few spills on the
// chain cost 2000 cycles a chunk.
constexpr uint32_t kLaunchRegs = 64, kChainRegs = 72, kSideRegs = 56;
static_assert(8 * kLaunchRegs * 32 <= 16384 && 4 * kChainRegs + 4 * kSideRegs <= 8 * kLaunchRegs, "register split");

// shared memory (bytes from a 1024-byte aligned base)
constexpr uint32_t kTile = 8192;                       // 64 rows x 128 bytes, 128-byte swizzle
constexpr uint32_t kHalf = 2 * kTile;                  // K then Q of 64 key channels
constexpr uint32_t kStageBytes = 2 * kHalf;
constexpr int kVStages = 1;
constexpr uint32_t SM_V = kStages * kStageBytes;       // V of the tile's columns 0-63, 64-127
constexpr uint32_t kVBytes = 2 * kTile;
constexpr uint32_t SM_T = SM_V + kVStages * kVBytes;       // T diag(beta) hi, lo
constexpr uint32_t SM_P = SM_T + 2 * kTile;            // P hi, lo
constexpr int kAP = 68;                                // fp32 row pitch of A (conflict-free 16-byte rows)
constexpr uint32_t SM_A = SM_P + 2 * kPRing * kTile;
constexpr uint32_t kABytes = kC * kAP * 4;
// per chunk: beta, e^b rk, rk e^(bC - b), e^b rq [64]; e^bC, whether mild, first token that is not finite
constexpr uint32_t SM_GATE = SM_A + 2 * kABytes;
constexpr uint32_t kGateFloats = 4 * kC + 4;
constexpr uint32_t SM_LOC = SM_GATE + kGRing * kGateFloats * 4;   // gate warps: two of rk, rq [64], b [64] (hi, lo), column factors [64]
constexpr uint32_t kLocFloats = 5 * kC;
constexpr uint32_t SM_OUT = SM_LOC + 2 * kLocFloats * 4;          // output warps: 8 token pairs x 32 columns each
constexpr uint32_t kOutPitch = 144;                               // a pair's 32 words, conflict-free 16-byte reads
constexpr uint32_t kSmem = SM_OUT + 4 * 8 * kOutPitch + 1024;     // + alignment slack
static_assert(kSmem <= 227 * 1024 - 1024, "shared memory");

// TMEM columns.  S holds for each quarter of the key rows its hi, then its lo terms,
// and is overwritten by the update D (fp32, as many columns) that the same
// chain warps read before they write the next S.
constexpr uint32_t TM_S = 0, TM_X = 128, TM_U = 192, TM_O = 256, TM_PU = 320, TM_G = 384;

struct Barriers {
    uint64_t full[kStages], empty[kStages], kq_ready[kStages], k_ready[kStages];
    uint64_t vfull[kVStages], vempty[kVStages];
    uint64_t work_full[kWorks], work_empty[kWorks];
    uint64_t s_ready, x_full, r_ready, u_full, u_ready, d_full, qs_full, o_full, o_free, t_ready;
    uint64_t g_full, g_free, a_ready[2], i_ready[2], a_free[2], scan_ready[2], p_ready[kPRing], p_free[kPRing], v_full, drain[3];
};

struct Params {
    const float *g, *beta;
    const void *v;
    __nv_bfloat16 *out;
    int N, Hk, Hv, Dv, tiles;
    int64_t chains;
    int pass;            // 0: whole sequences; 1, 2: the passes over segments
    GdnSegs segs;
    GdnTable tab;
    StateIO io;
    DevStatus *st;
    uint32_t wait_limit;
    Bounds bd;
};

// x0, x1 as two bf16 terms each, packed with x0 in the low halves.
__device__ __forceinline__ void split2(float x0, float x1, float &hi, float &lo)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&h);
    const float2 r = __fadd2_rn(make_float2(x0, x1),
                                make_float2(-__uint_as_float(u << 16), -__uint_as_float(u & 0xFFFF0000u)));
    const __nv_bfloat162 l = __floats2bfloat162_rn(r.x, r.y);
    hi = __uint_as_float(u);
    lo = __uint_as_float(*reinterpret_cast<const uint32_t *>(&l));
}

__device__ __forceinline__ bool bf16_finite(uint16_t x) { return (x & 0x7F80) != 0x7F80; }

__device__ __forceinline__ void mul2(float *x, float f0, float f1)
{
    const float2 y = __fmul2_rn(make_float2(x[0], x[1]), make_float2(f0, f1));
    x[0] = y.x;
    x[1] = y.y;
}

// x -= a (b0, b1)
__device__ __forceinline__ void fms2(float *x, float a, float b0, float b1)
{
    const float2 y = __ffma2_rn(make_float2(-a, -a), make_float2(b0, b1), make_float2(x[0], x[1]));
    x[0] = y.x;
    x[1] = y.y;
}

// Sum of two numbers held as two floats each (x the leading part): the exact
// error of the leading sum joins the small parts.
__device__ __forceinline__ float2 add_ff(float2 a, float2 b)
{
    const float s = a.x + b.x, bb = s - a.x;
    const float err = (a.x - (s - bb)) + (b.x - bb) + (a.y + b.y);
    const float hi = s + err;
    return make_float2(hi, err - (hi - s));
}

// Polls `bar` for phase `parity`; gives up after `limit` polls.
__device__ __forceinline__ bool wait_limited(uint64_t *bar, uint32_t parity, uint32_t limit)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, %3;\n\t"
        "POLL:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "add.u32 n, n, -1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@p bra DONE;\n\t"
        "@q bra POLL;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(limit)
        : "memory");
    return ok != 0;
}

constexpr uint32_t kDrainLimit = 1u << 22;

// NT tiles of 16 x 8 of a product of A's blocks, D = sign L R at columns 8 n[.]; K
// steps of 8 from k0[.] to k1, of at most KMAX.  All three in shared memory with A's row
// pitch; the tiles share L's rows and their split into terms.
template <int KMAX, int NT>
__device__ __forceinline__ void tile_product(const float *L, const float *R, float *D, const int (&n)[NT], const int (&k0)[NT],
                                             int k1, float sign, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    float d[NT][4], lo[NT][4];
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) d[u][q] = lo[u][q] = 0.f;
    L += g * kAP + t;
    R += t * kAP + g;
#pragma unroll 2   // (the roles share the schedulers' instruction caches: unrolled, long calls take 3 % more)
    for (int k = 0; k < KMAX; ++k)
        if (k < k1) {
            const float a[4] = {L[8 * k], L[8 * kAP + 8 * k], L[8 * k + 4], L[8 * kAP + 8 * k + 4]};
#pragma unroll
            for (int u = 0; u < NT; ++u)
                if (k >= k0[u]) {
                    const float b[2] = {R[8 * k * kAP + 8 * n[u]], R[(8 * k + 4) * kAP + 8 * n[u]]};
                    mma_tf32x3_apart(d[u], lo[u], a, b);
                }
        }
    D += g * kAP + 2 * t;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
        *reinterpret_cast<float2 *>(D + 8 * n[u]) = make_float2(sign * (d[u][0] + lo[u][0]), sign * (d[u][1] + lo[u][1]));
        *reinterpret_cast<float2 *>(D + 8 * kAP + 8 * n[u]) = make_float2(sign * (d[u][2] + lo[u][2]), sign * (d[u][3] + lo[u][3]));
    }
}

// Registers of a warpgroup (all of its warps call this, once).
template <uint32_t N> __device__ __forceinline__ void set_regs()
{
    if constexpr (N > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    if constexpr (N < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One chain as the roles see it.
enum Mode : int {
    kReal = 0,           // from its initial state, with outputs
    kOffset = 1,         // a segment from zeros, end state only
    kTransition = 2      // a segment from the identity with V = 0: its end state is the segment's transition
};
struct Chain {
    int n, h, tile;      // n < 0: no more work
    int t0, len, nch;    // of the segment
    int mode, seg, last; // last: the sequence ends in it
    int ckpt;            // first checkpoint slot of the sequence
};

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
gdn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv, const Params p)
{
    extern __shared__ uint8_t raw_sm[];
    __shared__ Barriers bar;
    __shared__ Chain works[kWorks];
    // columns in which a value was not finite, up to each chunk of its chain.  (A slot's last
    // readers, the outputs at their chain's end, are not more than three chunks behind: the
    // values of the fourth wait for the state update before them, and that for the outputs.)
    __shared__ uint32_t vbad[kVRing][4];
    __shared__ uint32_t tmem_sh;

    constexpr int HALVES = DK / 64;
    constexpr int SR = DK / 4;                  // key rows per chain thread
    uint8_t *sm = raw_sm + ((1024u - (smem_u32(raw_sm) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t limit = p.wait_limit;

    if (tid == 0) {
        // arrivals: one per warp of the role, or one of a commit or copy
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
            mbar_init(&bar.kq_ready[i], 4);
            mbar_init(&bar.k_ready[i], 4);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&bar.vfull[i], 1);
            mbar_init(&bar.vempty[i], 1);
        }
        for (int i = 0; i < kWorks; ++i) {
            mbar_init(&bar.work_full[i], 1);
            mbar_init(&bar.work_empty[i], kWorkReaders);
        }
        uint64_t *by16[] = {&bar.s_ready, &bar.r_ready, &bar.u_ready, &bar.t_ready,
                            &bar.a_free[0], &bar.a_free[1]};
        for (uint64_t *b : by16) mbar_init(b, kChainWarps);
        mbar_init(&bar.g_free, 4);
        mbar_init(&bar.o_free, 4);
        mbar_init(&bar.v_full, 2);
        for (int i = 0; i < 2; ++i) mbar_init(&bar.i_ready[i], 4);
        for (int i = 0; i < 2; ++i) mbar_init(&bar.a_ready[i], 2);
        for (int i = 0; i < kPRing; ++i) {
            mbar_init(&bar.p_ready[i], 2);
            mbar_init(&bar.p_free[i], 1);
        }
        uint64_t *by1[] = {&bar.x_full, &bar.u_full, &bar.d_full, &bar.qs_full, &bar.o_full, &bar.g_full, &bar.scan_ready[0],
                           &bar.scan_ready[1], &bar.drain[0], &bar.drain[1], &bar.drain[2]};
        for (uint64_t *b : by1) mbar_init(b, 1);
        fence_mbar_init();
    }
    // the status of the offsets (CTAs whose waits give up report to the same word, which was
    // cleared before the launch: in whatever order, the first report stays)
    if (warp == 1 && blockIdx.x == 0 && !p.tab.cu) gdn_sequence<false>(p.tab, 0, p.st);
    if (warp == 0) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = tmem_sh;

    bool alive = true;
    // a wait of whole warps: the same answer in every lane
    auto wait_w = [&](uint64_t *b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_limited(b, parity, limit));
    };
    // one arrival of a warp, after everything its lanes did
    auto arrive_w = [&](uint64_t *b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(b);
    };
    // the k-th chain of this CTA (false: gave up waiting for it)
    auto get_work = [&](int k, Chain &w) -> bool {
        const int slot = k % kWorks;
        if (!wait_w(&bar.work_full[slot], (k / kWorks) & 1)) return false;
        w = works[slot];
        arrive_w(&bar.work_empty[slot]);
        return true;
    };

    // never leaves an MMA of this warp in flight
    auto drain_mma = [&](int i) {
        if (elect_one()) mma_commit(&bar.drain[i]);
        __syncwarp();
        mbar_wait_bounded(&bar.drain[i], 0, kDrainLimit);
    };

    if (warp >= kProducerWarp) {
        set_regs<kSideRegs>();
        if (warp == kProducerWarp) {
            // ------------------------------------------------------------ producer
            int cc = 0;
            // the chain of number id: n < 0 behind the last; false: there is no such
            // segment (the sequence is shorter)
            auto chain_of = [&](int64_t id, Chain &w) -> bool {
                w = Chain{-1, 0, 0, 0, 0, 0, kReal, 0, 1, 0};
                int64_t place;
                if (id >= p.chains) return true;
                const int tiles = p.Hv * p.tiles;
                if (p.pass == 0) {
                    place = id / tiles;
                } else {
                    // pass 1: segments 0 .. P - 2, then the transitions of 1 .. P - 2; pass 2: 1 .. P - 1
                    const int P = p.segs.P, per = tiles * (P - 1) + (p.pass == 1 ? p.Hv * (P - 2) : 0);
                    place = id / per;
                    id %= per;
                    if (id < (int64_t)tiles * (P - 1)) {
                        w.seg = (int)(id / tiles) + (p.pass == 2);
                        w.mode = p.pass == 1 && w.seg > 0 ? kOffset : kReal;
                    } else {
                        id -= (int64_t)tiles * (P - 1);
                        w.seg = (int)(id / p.Hv) + 1;
                        w.mode = kTransition;
                    }
                }
                if (w.mode == kTransition) {
                    w.h = (int)(id % p.Hv);
                } else {
                    w.h = (int)(id % tiles) / p.tiles;
                    w.tile = (int)(id % tiles) % p.tiles;
                }
                const GdnSeq seq = gdn_sequence(p.tab, (int)place, nullptr);
                w.n = seq.n;
                w.ckpt = seq.ckpt;
                const int len = seq.len, at = w.seg * p.segs.G * kC;
                if (w.seg > 0 && at >= len) return false;
                w.t0 = seq.t0 + at;
                w.len = len - at;
                if (p.pass != 0 && w.seg < p.segs.P - 1 && w.len > p.segs.G * kC) {
                    w.len = p.segs.G * kC;
                    w.last = 0;
                }
                if (w.mode != kReal && w.last) return false;   // (nothing starts from its end)
                w.len = dbg_rows(w.t0, w.len, p.bd);
                w.nch = (w.len + kC - 1) / kC;
                return true;
            };
            // V of a chunk is asked for after K and Q of the next: its only stage is free late,
            // once T V of the chunk before was formed, and K and Q are wanted early
            int v_tile = 0, v_h = 0, v_t = 0, v_asked = 0;
            auto values = [&](int c) -> bool {
                const int vs = c % kVStages;
                if (c >= kVStages && !wait_w(&bar.vempty[vs], (c / kVStages - 1) & 1)) return false;
                if (elect_one()) {
                    const uint32_t dvb = min(2u, (uint32_t)(p.Dv - 128 * v_tile) / 64);
                    uint8_t *vt = sm + SM_V + vs * kVBytes;
                    mbar_arrive_expect_tx(&bar.vfull[vs], dvb * kTile);
                    tma_load_3d(vt, &mv, 128 * v_tile, v_h, v_t, &bar.vfull[vs]);
                    if (dvb > 1) tma_load_3d(vt + kTile, &mv, 128 * v_tile + 64, v_h, v_t, &bar.vfull[vs]);
                }
                __syncwarp();
                v_asked = c + 1;
                return true;
            };
            int64_t id = blockIdx.x;
            for (int k = 0; alive;) {
                Chain w;
                const bool there = chain_of(id, w);
                int32_t more = 0;
                if (lane == 0 && w.n >= 0 && p.tab.cu) more = atomicAdd(p.tab.next + (p.pass == 2), 1);
                id = (int64_t)gridDim.x + __shfl_sync(0xffffffffu, more, 0);
                if (!there) continue;
                // (before chains without a chunk: their slots may wait for the last chunk's chain)
                if ((w.n < 0 || w.nch == 0) && v_asked < cc && !values(cc - 1)) {
                    alive = false;
                    break;
                }
                const int slot = k % kWorks;
                if (k >= kWorks && !wait_w(&bar.work_empty[slot], (k / kWorks - 1) & 1)) {
                    alive = false;
                    break;
                }
                if (lane == 0) {
                    works[slot] = w;
                    mbar_arrive(&bar.work_full[slot]);
                }
                __syncwarp();
                ++k;
                if (w.n < 0) break;
                const int hk = w.h / (p.Hv / p.Hk);
                for (int c = 0; c < w.nch; ++c, ++cc) {
                    const int s = cc % kStages, t = w.t0 + c * kC;
                    if (cc >= kStages && !wait_w(&bar.empty[s], (cc / kStages - 1) & 1)) {
                        alive = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *stg = sm + s * kStageBytes;
                        mbar_arrive_expect_tx(&bar.full[s], 2 * HALVES * kTile);
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf) {
                            tma_load_3d(stg + hf * kHalf, &mk, 64 * hf, hk, t, &bar.full[s]);
                            tma_load_3d(stg + hf * kHalf + kTile, &mq, 64 * hf, hk, t, &bar.full[s]);
                        }
                    }
                    __syncwarp();
                    if (v_asked < cc && !values(cc - 1)) {
                        ++cc;
                        alive = false;
                        break;
                    }
                    v_tile = w.tile;
                    v_h = w.h;
                    v_t = t;
                }
            }
            if (alive && v_asked < cc) alive = values(cc - 1);
            // never leave a copy in flight
            for (int c = max(0, cc - kStages); c < cc; ++c)
                mbar_wait_bounded(&bar.full[c % kStages], (c / kStages) & 1, kDrainLimit);
            for (int c = max(0, v_asked - kVStages); c < v_asked; ++c)
                mbar_wait_bounded(&bar.vfull[c % kVStages], (c / kVStages) & 1, kDrainLimit);
        } else if (warp == kIssuerWarp) {
            // ------------------------------------------------------------ issuer
            int cc = 0;
            constexpr uint32_t id_dk = idesc_bf16(128, DK) | kIdescBMn;
            // column of key rows 16 r .. 16 r + 15 of S, hi term
            auto s_column = [](int r) -> uint32_t { return TM_S + 16 * r / SR * SR + 16 * r % SR / 2; };
            Chain w;
            for (int k = 0; alive; ++k) {
                if (!get_work(k, w)) { alive = false; break; }
                if (w.n < 0) break;
                for (int c = 0; c < w.nch; ++c, ++cc) {
                    const int s = cc % kStages, pr = cc % kPRing;
                    const uint32_t stg = sb + s * kStageBytes, ph = cc & 1;
                    // X = K S (both terms of S); the previous chunk's P U has read the columns of X
                    if (!wait_w(&bar.k_ready[s], (cc / kStages) & 1) || !wait_w(&bar.s_ready, ph) ||
                        (cc > 0 && !wait_w(&bar.o_full, ph ^ 1))) {
                        alive = false;
                        break;
                    }
                    fence_after_sync();
                    constexpr uint32_t id64 = idesc_bf16(128, 64);
                    if (elect_one()) {
#pragma unroll 1
                        for (int u = 0; u < 2 * HALVES; ++u) {
                            const uint64_t d = make_desc_sw128(stg + (u % HALVES) * kHalf, 16);
                            const uint32_t a = tm + s_column(4 * (u % HALVES)) + (u < HALVES ? 0 : SR / 2);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) mma_f16_ts(tm + TM_X, a + s_column(ks), d + 2 * ks, id64, u + ks > 0);
                        }
                        mma_commit(&bar.x_full);
                    }
                    __syncwarp();
                    // U += T diag(beta) X, X = -e^b rk K S: X hi T hi, X hi T lo, X lo T hi
                    if (!wait_w(&bar.v_full, ph) || !wait_w(&bar.r_ready, ph)) { alive = false; break; }
                    fence_after_sync();
                    if (elect_one()) {
#pragma unroll 1
                        for (int t = 0; t < 3; ++t) {
                            const uint64_t d = make_desc_sw128(sb + SM_T + (t == 1 ? kTile : 0), 16);
                            const uint32_t a = tm + TM_X + (t == 2 ? 8 : 0);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ts(tm + TM_U + 16 * ks, a + 16 * ks, d + 130 * ks, idesc_bf16(128, 64 - 16 * ks), 1);
                        }
                        mma_commit(&bar.u_full);
                    }
                    __syncwarp();
                    // Q S (both terms of S), once the previous outputs were read
                    if (cc > 0 && !wait_w(&bar.o_free, ph ^ 1)) { alive = false; break; }
                    fence_after_sync();
                    if (elect_one()) {
#pragma unroll 1
                        for (int u = 0; u < 2 * HALVES; ++u) {
                            const uint64_t d = make_desc_sw128(stg + kTile + (u % HALVES) * kHalf, 16);
                            const uint32_t a = tm + s_column(4 * (u % HALVES)) + (u < HALVES ? 0 : SR / 2);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) mma_f16_ts(tm + TM_O, a + s_column(ks), d + 2 * ks, id64, u + ks > 0);
                        }
                        mma_commit(&bar.qs_full);
                    }
                    __syncwarp();
                    // D = K^T (scaled U), both terms, over S
                    if (!wait_w(&bar.u_ready, ph) || !wait_w(&bar.qs_full, ph)) { alive = false; break; }
                    fence_after_sync();
                    if (elect_one()) {
#pragma unroll 1
                        for (int t = 0; t < 2; ++t) {
                            const uint64_t d = make_desc_sw128(stg, kHalf);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ts(tm + TM_S, tm + TM_U + 16 * ks + 8 * t, d + 128 * ks, id_dk, t + ks > 0);
                        }
                        mma_commit(&bar.d_full);
                        mma_commit(&bar.empty[s]);
                    }
                    __syncwarp();
                    // P U, lower triangular as T: P hi U hi, P hi U lo, P lo U hi
                    if (!wait_w(&bar.p_ready[pr], (cc / kPRing) & 1)) { alive = false; break; }
                    fence_after_sync();
                    if (elect_one()) {
#pragma unroll 1
                        for (int t = 0; t < 3; ++t) {
                            const uint64_t d = make_desc_sw128(sb + SM_P + (2 * pr + (t == 2)) * kTile, 16);
                            const uint32_t a = tm + TM_X + (t == 1 ? 8 : 0);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ts(tm + TM_PU + 16 * ks, a + 16 * ks, d + 130 * ks,
                                           idesc_bf16(128, 64 - 16 * ks), t + ks > 0);
                        }
                        mma_commit(&bar.o_full);
                        mma_commit(&bar.p_free[pr]);
                    }
                    __syncwarp();
                }
            }
            drain_mma(0);
        } else if (warp == kGramWarp) {
            // ------------------------------------------------------------ G
            // and, a chunk ahead of the gate warps, the running decays
            int cc = 0;
            Chain w{};
            // of chunk c of w, the cc-th: the buffers are those of chunk cc - 2, whose G was
            // read, and of chunk cc - kGRing, whose state update was (P of chunk cc - 2 waited
            // for the products of chunk cc - 2 - kPRing)
            auto scan = [&](int c, int cc) {
                const int L = min(kC, w.len - c * kC);
                const int64_t tok = (int64_t)(w.t0 + c * kC) * p.Hv + w.h;
                float g0 = 0.f, g1 = 0.f;
                float2 bt = make_float2(0.f, 0.f);
                const int64_t at = tok + (int64_t)(2 * lane) * p.Hv;
                if (2 * lane < L) {
                    g0 = p.g[at];
                    bt.x = p.beta[at];
                }
                if (2 * lane + 1 < L) {
                    g1 = p.g[at + p.Hv];
                    bt.y = p.beta[at + p.Hv];
                }
                // gates that are not finite (but -inf, a decay): zeros, and the first one's token
                const bool bad0 = !(g0 < INFINITY && fabsf(bt.x) < INFINITY), bad1 = !(g1 < INFINITY && fabsf(bt.y) < INFINITY);
                const uint32_t m0 = __ballot_sync(0xffffffffu, bad0), m1 = __ballot_sync(0xffffffffu, bad1);
                if (bad0) g0 = bt.x = 0.f;
                if (bad1) g1 = bt.y = 0.f;
                float *loc = reinterpret_cast<float *>(sm + SM_LOC) + (cc & 1) * kLocFloats, *bb = loc + 2 * kC;
                float *gate = reinterpret_cast<float *>(sm + SM_GATE) + (cc % kGRing) * kGateFloats;
                // running sums in units of log2, as two floats (hi + lo, 48 bits):
                // differences of far positions keep their low bits.  -inf and
                // anything below -1024 a token clear the state alike (2^-1024 is 0).
                constexpr float kL = 1.4426950408889634f, kLlo = (float)(1.4426950408889634 - (double)kL);
                g0 = fmaxf(g0, -1024.f);
                g1 = fmaxf(g1, -1024.f);
                const float h0 = g0 * kL, h1 = g1 * kL;
                const float2 x0 = make_float2(h0, fmaf(g0, kL, -h0) + g0 * kLlo);
                const float2 x1 = make_float2(h1, fmaf(g1, kL, -h1) + g1 * kLlo);
                float2 b1 = add_ff(x0, x1);
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const float2 y = make_float2(__shfl_up_sync(0xffffffffu, b1.x, o), __shfl_up_sync(0xffffffffu, b1.y, o));
                    if (lane >= o) b1 = add_ff(b1, y);
                }
                const float2 b0 = add_ff(b1, make_float2(-x1.x, -x1.y));
                const float2 bc = make_float2(__shfl_sync(0xffffffffu, b1.x, 31), __shfl_sync(0xffffffffu, b1.y, 31));
                *reinterpret_cast<float4 *>(bb + 4 * lane) = make_float4(b0.x, b0.y, b1.x, b1.y);
                // e^b and e^(b_C - b), still without the norms
                *reinterpret_cast<float2 *>(gate + kC + 2 * lane) = make_float2(ex2_ftz(b0.x), ex2_ftz(b1.x));
                *reinterpret_cast<float2 *>(gate + 2 * kC + 2 * lane) =
                    make_float2(ex2_ftz((bc.x - b0.x) + (bc.y - b0.y)), ex2_ftz((bc.x - b1.x) + (bc.y - b1.y)));
                // e^(b at the end of the token's 16 - b): the decay of a column to the
                // end of its block
                const int e16 = lane | 7;
                const float2 be = make_float2(__shfl_sync(0xffffffffu, b1.x, e16), __shfl_sync(0xffffffffu, b1.y, e16));
                *reinterpret_cast<float2 *>(loc + 4 * kC + 2 * lane) =
                    make_float2(ex2_ftz((be.x - b0.x) + (be.y - b0.y)), ex2_ftz((be.x - b1.x) + (be.y - b1.y)));
                *reinterpret_cast<float2 *>(gate + 2 * lane) = bt;
                // mild: no block of 16 decays by more than 2^-32, so that decays inside a block may
                // go by its end as well (an exponent up to 32 is off by 2^-20 at most)
                const bool mild = __all_sync(0xffffffffu, b0.x - be.x <= 32.f);
                if (lane == 0) {
                    gate[4 * kC] = ex2_ftz(bc.x);
                    gate[4 * kC + 1] = mild ? 1.f : 0.f;
                    reinterpret_cast<int *>(gate)[4 * kC + 2] =
                        min(m0 ? 2 * __ffs(m0) - 2 : kC, m1 ? 2 * __ffs(m1) - 1 : kC);
                }
                arrive_w(&bar.scan_ready[cc & 1]);
            };
            for (int k = 0; alive; ++k) {
                if (!get_work(k, w)) { alive = false; break; }
                if (w.n < 0) break;
                if (w.nch > 0) scan(0, cc);
                for (int c = 0; c < w.nch; ++c, ++cc) {
                    // its tiles have landed and the last G was read
                    if (!wait_w(&bar.kq_ready[cc % kStages], (cc / kStages) & 1) || (cc > 0 && !wait_w(&bar.g_free, (cc - 1) & 1))) {
                        alive = false;
                        break;
                    }
                    fence_after_sync();
                    if (elect_one()) {
                        const uint32_t stg = sb + (cc % kStages) * kStageBytes;
#pragma unroll 1
                        for (int hf = 0; hf < HALVES; ++hf) {
                            const uint64_t d = make_desc_sw128(stg + hf * kHalf, 16);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) mma_bf16(tm + TM_G, d + 2 * ks, d + 2 * ks, idesc_bf16(128, 64), hf + ks > 0);
                        }
                        mma_commit(&bar.g_full);
                    }
                    __syncwarp();
                    if (c + 1 < w.nch) scan(c + 1, cc + 1);
                }
            }
            drain_mma(1);
        } else if (warp == kValueWarp) {
            // ------------------------------------------------------------ T V
            // U = T diag(beta) V, the part of a chunk's U that does not wait for the
            // state, once the previous chunk's state update has read the columns of U;
            // T is lower triangular, so K step ks reaches rows 16 ks .. 63 only
            int cc = 0;
            Chain w;
            for (int k = 0; alive; ++k) {
                if (!get_work(k, w)) { alive = false; break; }
                if (w.n < 0) break;
                // its initial state into L2, a chunk before it is read (the first chain's is
                // read at once)
                if (k > 0 && p.io.init && w.mode == kReal && w.seg == 0) {
                    const int64_t slot = pool_slot(p.io.init_slots, w.n, p.io.pool);
                    if (slot >= 0 && dbg_in(slot, p.bd.states, kDbgState)) {
                        const int lines = min(128, p.Dv - 128 * w.tile) / 32, col = 32 * (lane & 3);
                        const float *src = p.io.init + ((slot * p.Hv + w.h) * DK + (lane >> 2)) * p.Dv + 128 * w.tile + col;
#pragma unroll 1
                        for (int i = 0; i < DK && (lane & 3) < lines; i += 8, src += 8 * (int64_t)p.Dv) prefetch_line_l2(src);
                        __syncwarp();
                    }
                }
                uint32_t dead = 0;   // of the lane's columns lane + 32 i, those with a value that is not finite
                for (int c = 0; c < w.nch; ++c, ++cc) {
                    const int vs = cc % kVStages, L = w.mode == kTransition ? 0 : w.len - c * kC;
                    if (!wait_w(&bar.vfull[vs], (cc / kVStages) & 1)) { alive = false; break; }
                    // rows behind the sequence's end belong to another sequence (or to nobody)
                    // and must be zero
                    if (L < kC) {
                        for (int u = lane + 8 * L; u < 8 * kC; u += 32) {
                            uint8_t *vr = sm + SM_V + vs * kVBytes + 16 * u;
                            *reinterpret_cast<uint4 *>(vr) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(vr + kTile) = make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();
                        __syncwarp();
                    }
                    // 0 x: not a number for every value that is not finite
                    const int cols = L > 0 ? min(128, p.Dv - 128 * w.tile) : 0;
                    bool bad = false;
                    {
                        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
                        __nv_bfloat162 z[2] = {zero, zero};
#pragma unroll 4
                        for (int u = lane; u < 8 * cols; u += 32) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(sm + SM_V + vs * kVBytes + 16 * u);
                            const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                z[m & 1] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&e[m]), zero, z[m & 1]);
                        }
                        z[0] = __hadd2(z[0], z[1]);
                        bad = __any_sync(0xffffffffu, dead != 0 || __hisnan(z[0].x) || __hisnan(z[0].y));
                    }
                    uint32_t words = 0;
                    if (bad) {
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            const int col = lane + 32 * i;
#pragma unroll 1
                            for (int r = 0; r < (col < cols ? min(L, kC) : 0); ++r) {
                                uint16_t *at = reinterpret_cast<uint16_t *>(sm + SM_V + vs * kVBytes + (col >> 6) * kTile + r * 128 +
                                                                            ((((col & 63) >> 3) ^ (r & 7)) * 16) + (col & 7) * 2);
                                if (!bf16_finite(*at)) {
                                    *at = 0;
                                    dead |= 1u << i;
                                }
                            }
                            const uint32_t word = __ballot_sync(0xffffffffu, dead >> i & 1);
                            if (lane == i) words = word;
                        }
                        fence_async_smem();
                    }
                    if (lane < 4) vbad[cc % kVRing][lane] = words;
                    __syncwarp();
                    if (!wait_w(&bar.t_ready, cc & 1) || (cc > 0 && !wait_w(&bar.d_full, (cc - 1) & 1))) {
                        alive = false;
                        break;
                    }
                    fence_after_sync();
                    if (elect_one()) {
                        const uint32_t vt = sb + SM_V + vs * kVBytes;
#pragma unroll 1
                        for (int t = 0; t < 2; ++t) {
                            const uint64_t a = make_desc_sw128(vt, kTile), d = make_desc_sw128(sb + SM_T + t * kTile, 16);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_bf16(tm + TM_U + 16 * ks, a + 128 * ks, d + 130 * ks, idesc_bf16(128, 64 - 16 * ks) | kIdescAMn,
                                         t + ks > 0);
                        }
                        mma_commit(&bar.v_full);
                        mma_commit(&bar.vempty[vs]);
                        // (an arrival of its own: vbad is seen behind v_full)
                        mbar_arrive(&bar.v_full);
                    }
                    __syncwarp();
                }
            }
            drain_mma(2);
        }
    } else if (warp >= kOutWarp0) {
        // ------------------------------------------------------------ outputs
        // O = e^b rq (Q S) + P U; a warp takes 32 columns (its TMEM lanes), 16 tokens at a
        // time.  Token pairs go as words through a tile of the warp's own, so that each lane
        // stores 16 bytes of two tokens.
        set_regs<kSideRegs>();
        const int q4 = warp & 3, pair = lane >> 2, c8 = 8 * (lane & 3);
        const uint32_t lb = tm + ((uint32_t)(32 * q4) << 16);
        uint8_t *tile = sm + SM_OUT + q4 * 8 * kOutPitch;
        int cc = 0;
        Chain w;
        for (int k = 0; alive; ++k) {
            if (!get_work(k, w)) { alive = false; break; }
            if (w.n < 0) break;
            const int col = 128 * w.tile + 32 * q4 + c8;
            const bool store = w.mode == kReal && col < p.Dv;   // (of the whole warp: Dv is a multiple of 32)
            for (int c = 0; c < w.nch; ++c, ++cc) {
                if (!wait_w(&bar.o_full, cc & 1)) { alive = false; break; }
                if (!store) {
                    arrive_w(&bar.o_free);
                    continue;
                }
                fence_after_sync();
                const float *f = reinterpret_cast<const float *>(sm + SM_GATE) + (cc % kGRing) * kGateFloats + 3 * kC;
#pragma unroll 1
                for (int i = 0; i < kC; i += 16) {
                    float x[16], y[16];
                    tmem_ld16(lb + TM_O + i, x);
                    tmem_ld16(lb + TM_PU + i, y);
                    tmem_ld_wait();
                    if (i == kC - 16) {
                        fence_before_sync();
                        arrive_w(&bar.o_free);
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 e = *reinterpret_cast<const float4 *>(f + i + j);
                        const float2 o0 = __ffma2_rn(make_float2(e.x, e.y), make_float2(x[j], x[j + 1]), make_float2(y[j], y[j + 1]));
                        const float2 o1 = __ffma2_rn(make_float2(e.z, e.w), make_float2(x[j + 2], x[j + 3]),
                                                     make_float2(y[j + 2], y[j + 3]));
                        const __nv_bfloat162 v0 = __floats2bfloat162_rn(o0.x, o0.y), v1 = __floats2bfloat162_rn(o1.x, o1.y);
                        uint8_t *at = tile + j / 2 * kOutPitch + 4 * lane;
                        *reinterpret_cast<uint32_t *>(at) = *reinterpret_cast<const uint32_t *>(&v0);
                        *reinterpret_cast<uint32_t *>(at + kOutPitch) = *reinterpret_cast<const uint32_t *>(&v1);
                    }
                    __syncwarp();
                    const uint4 u = *reinterpret_cast<const uint4 *>(tile + pair * kOutPitch + 4 * c8);
                    const uint4 v = *reinterpret_cast<const uint4 *>(tile + pair * kOutPitch + 4 * c8 + 16);
                    const int t = kC * c + i + 2 * pair, left = w.len - t;
                    __nv_bfloat16 *dst = p.out + ((int64_t)(w.t0 + t) * p.Hv + w.h) * p.Dv + col;
                    if (left > 0)
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.z, u.w, 0x5410),
                                                                     __byte_perm(v.x, v.y, 0x5410), __byte_perm(v.z, v.w, 0x5410));
                    if (left > 1)
                        *reinterpret_cast<uint4 *>(dst + (int64_t)p.Hv * p.Dv) =
                            make_uint4(__byte_perm(u.x, u.y, 0x7632), __byte_perm(u.z, u.w, 0x7632),
                                       __byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x7632));
                    __syncwarp();
                }
            }
            // over them, what follows a value that is not finite in its column
            if (alive && w.nch > 0 && w.mode == kReal && (vbad[(cc - 1) % kVRing][q4] >> lane & 1)) {
                const int64_t at = ((int64_t)w.t0 * p.Hv + w.h) * p.Dv + 128 * w.tile + 32 * q4 + lane, step = (int64_t)p.Hv * p.Dv;
                const uint16_t *v = reinterpret_cast<const uint16_t *>(p.v) + at;
                bool seen = false;
#pragma unroll 1
                for (int64_t t = 0; t < w.len; ++t) {
                    seen |= !bf16_finite(v[t * step]);
                    if (seen) p.out[at + t * step] = __float2bfloat16(NAN);
                }
            }
            __syncwarp();
        }
    } else if (warp >= kInvWarp0) {
        // ------------------------------------------------------------ inverse
        // T = (I + A)^-1 in place over A (fp32, lower triangle): the 16 x 16 diagonal
        // blocks, then merged to blocks of 32 and to the whole
        set_regs<kSideRegs>();
        const int wi = warp - kInvWarp0;
        int cc = 0;
        Chain w;
        for (int k = 0; alive; ++k) {
            alive = named_bar_and(2, 128, get_work(k, w));
            if (!alive || w.n < 0) break;
            for (int c = 0; c < w.nch && alive; ++c, ++cc) {
                // the group's barriers need all of it: every wait is answered in common
                alive = named_bar_and(2, 128, wait_w(&bar.a_ready[cc & 1], (cc >> 1) & 1));
                if (!alive) break;
                float *A = reinterpret_cast<float *>(sm + SM_A + (cc & 1) * kABytes);
                if (wi < 2) {
                    // diagonal blocks of 16, two a warp: T (I + A) = I by columns from the
                    // right, lane r row r of T: T[r][k] is final once the columns right of k
                    // were subtracted, so the chain is one multiply-add per column
                    float *blk = A + (32 * wi + (lane & 16)) * (kAP + 1);
                    const int r = lane & 15;
                    float x[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = j == r ? 1.f : 0.f;
#pragma unroll
                    for (int k = 15; k > 0; --k) {
#pragma unroll
                        for (int j = 0; j < k; j += 4) {
                            const float4 a = *reinterpret_cast<const float4 *>(blk + k * kAP + j);
                            fms2(x + j, x[k], a.x, a.y);       // (A is zero on and above its diagonal)
                            if (j + 2 < k) fms2(x + j + 2, x[k], a.z, a.w);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(blk + r * kAP + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                }
                named_bar(2, 128);
                // merges T21 = -(T22 A21) T11 on warp-level products of tf32 terms, for the
                // blocks of 32 and then for the whole; the left product goes above the
                // diagonal, where nothing else is
                {
                    float *B = A + 32 * (wi >> 1) * (kAP + 1);
                    const int n[1] = {wi & 1}, from[1] = {0};
                    tile_product<2>(B + 16 * (kAP + 1), B + 16 * kAP, B + 16, n, from, 2, 1.f, lane);
                    named_bar(2, 128);
                    tile_product<2>(B + 16, B, B + 16 * kAP, n, n, 2, -1.f, lane);
                }
                named_bar(2, 128);
                {
                    // 16 rows and two of four tiles of 8 columns a warp
                    const int r0 = 16 * (wi & 1), n[2] = {wi >> 1, 3 - (wi >> 1)}, from[2] = {0, 0};
                    tile_product<4>(A + (32 + r0) * kAP + 32, A + 32 * kAP, A + r0 * kAP + 32, n, from, 2 + 2 * (wi & 1), 1.f, lane);
                    named_bar(2, 128);
                    tile_product<4>(A + r0 * kAP + 32, A, A + (32 + r0) * kAP, n, n, 4, -1.f, lane);
                }
                arrive_w(&bar.i_ready[cc & 1]);
            }
        }
    } else if (warp >= kGateWarp0) {
        // ------------------------------------------------------------ gates
        set_regs<kSideRegs>();
        const int wa = warp - kGateWarp0, t = tid - 32 * kGateWarp0, i = t & 63;
        const bool krow = t < 64;
        const uint32_t lb = tm + ((uint32_t)(32 * wa) << 16) + TM_G;
        int cc = 0;
        Chain w;
        for (int k = 0; alive; ++k) {
            alive = named_bar_and(1, 128, get_work(k, w));
            if (!alive || w.n < 0) break;
            for (int c = 0; c < w.nch && alive; ++c, ++cc) {
                const int s = cc % kStages, L = min(kC, w.len - c * kC);
                float *loc = reinterpret_cast<float *>(sm + SM_LOC) + (cc & 1) * kLocFloats;
                float *rk = loc, *bb = loc + 2 * kC;   // rk, rq; b as pairs (hi, lo)
                float *gate = reinterpret_cast<float *>(sm + SM_GATE) + (cc % kGRing) * kGateFloats;
                // the group's barriers need all of it: every wait is answered in common
                alive = named_bar_and(1, 128, wait_w(&bar.full[s], (cc / kStages) & 1) &&
                                                  wait_w(&bar.scan_ready[cc & 1], (cc >> 1) & 1));
                if (!alive) break;
                uint8_t *row = sm + s * kStageBytes + t * 128;   // K rows, then Q rows
                // rows behind the sequence's end belong to another sequence (or to
                // nobody): K is an operand there, and must be zero
                if (L < kC) {
                    if (krow && i >= L) {
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4 *>(row + hf * kHalf + 16 * q) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                arrive_w(&bar.kq_ready[s]);
                float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll 4
                    for (int q = 0; q < 8; ++q) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(row + hf * kHalf + ((q ^ (t & 7)) * 16));
                        const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const float2 x = make_float2(__uint_as_float(e[m] << 16), __uint_as_float(e[m] & 0xFFFF0000u));
                            ss2 = __ffma2_rn(x, x, ss2);
                        }
                    }
                const float ss = ss2.x + ss2.y + 1e-6f;
                // 0 behind the end, and for a row whose square is not finite
                const float r = i < L && ss < INFINITY ? rsqrtf(ss) : 0.f;
                const uint32_t bad = __ballot_sync(0xffffffffu, krow && i < L && r == 0.f);
                if (bad && lane == 0) atomicMin(reinterpret_cast<int *>(gate) + 4 * kC + 2, 32 * wa + __ffs(bad) - 1);
                const float eq = gate[kC + i] * r;       // (of the queries)
                loc[t] = r;                              // rk, then rq
                if (krow) {
                    gate[2 * kC + i] *= r;
                    loc[4 * kC + i] *= r;                // column factor of the blocks below the diagonal
                }
                named_bar(1, 128);   // e^b was read for the queries before it becomes e^b rk
                const int from = reinterpret_cast<const int *>(gate)[4 * kC + 2];
                if (krow) gate[kC + i] *= r;
                else gate[3 * kC + i] = i < from ? eq : NAN;
                if (t == 0 && from < kC) gate[4 * kC] = NAN;

                // A's rows wait for T of two chunks ago to be taken from there, P's for the
                // products that read it
                bool ok = wait_w(&bar.g_full, cc & 1);
                if (krow && cc >= 2) ok = ok && wait_w(&bar.a_free[cc & 1], ((cc >> 1) - 1) & 1);
                if (!krow && cc >= kPRing) ok = ok && wait_w(&bar.p_free[cc % kPRing], (cc / kPRing - 1) & 1);
                alive = named_bar_and(1, 128, ok);
                if (!alive) break;
                fence_after_sync();
                // (G, which had them, is masked below)
                if (from < kC) {
                    if (krow && i < L && r == 0.f) {
#pragma unroll 1
                        for (int q = 0; q < 8 * HALVES; ++q)
                            *reinterpret_cast<uint4 *>(row + (q >> 3) * kHalf + 16 * (q & 7)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                arrive_w(&bar.k_ready[s]);
                // the row's last column; none of a key that is not finite, or behind one
                const int diag = krow ? (i < from ? i - 1 : -1) : min(i, from - 1);
                const float2 bi = *reinterpret_cast<const float2 *>(bb + 2 * i);
                const float rc = krow ? gate[i] * r : r;
                const bool mild = gate[4 * kC + 1] != 0.f;
                float *arow = reinterpret_cast<float *>(sm + SM_A + (cc & 1) * kABytes) + i * kAP;
                uint8_t *prow = sm + SM_P + (cc % kPRing) * 2 * kTile + i * 128;
                const int first = (wa & 1) ? 32 : 0;     // the warp's first row: columns below it are all kept
#pragma unroll 1
                for (int j16 = 0; j16 < first + 32; j16 += 16) {
                    float x[16];
                    tmem_ld16(lb + j16, x);
                    const int last = diag - j16;
                    if (mild || j16 < first) {
                        // e^(b_i - b_j) as the decay from the block's end to row i times that of
                        // column j to the end; left of the warp's rows both are <= 1 however
                        // strong the decay, in a row's own block the first is up to 2^32
                        const float2 be = *reinterpret_cast<const float2 *>(bb + 2 * (j16 + 15));
                        const float f = rc * ex2_ftz((bi.x - be.x) + (bi.y - be.y));
                        tmem_ld_wait();
#pragma unroll
                        for (int j4 = 0; j4 < 16; j4 += 4) {
                            const float4 cj = *reinterpret_cast<const float4 *>(loc + 4 * kC + j16 + j4);
                            mul2(x + j4, cj.x, cj.y);
                            mul2(x + j4 + 2, cj.z, cj.w);
                            mul2(x + j4, f, f);
                            mul2(x + j4 + 2, f, f);
                        }
                    } else {
                        // the 32 columns around the diagonal, each decay by itself
                        tmem_ld_wait();
#pragma unroll
                        for (int j2 = 0; j2 < 16; j2 += 2) {
                            const float4 bj = *reinterpret_cast<const float4 *>(bb + 2 * (j16 + j2));
                            const float2 rr = *reinterpret_cast<const float2 *>(rk + j16 + j2);
                            const float2 d0 = __fadd2_rn(bi, make_float2(-bj.x, -bj.y)), d1 = __fadd2_rn(bi, make_float2(-bj.z, -bj.w));
                            mul2(x + j2, rr.x, rr.y);
                            mul2(x + j2, rc, rc);
                            mul2(x + j2, ex2_ftz(d0.x + d0.y), ex2_ftz(d1.x + d1.y));
                        }
                    }
                    if (j16 >= first || from < kC) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = j <= last ? x[j] : 0.f;
                    }
                    if (krow) {
#pragma unroll
                        for (int j4 = 0; j4 < 16; j4 += 4)
                            *reinterpret_cast<float4 *>(arow + j16 + j4) = make_float4(x[j4], x[j4 + 1], x[j4 + 2], x[j4 + 3]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float hi[4], lo[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m) split2(x[8 * q + 2 * m], x[8 * q + 2 * m + 1], hi[m], lo[m]);
                            uint8_t *dst = prow + (((j16 / 8 + q) ^ (i & 7)) * 16);
                            *reinterpret_cast<float4 *>(dst) = make_float4(hi[0], hi[1], hi[2], hi[3]);
                            *reinterpret_cast<float4 *>(dst + kTile) = make_float4(lo[0], lo[1], lo[2], lo[3]);
                        }
                    }
                }
                fence_before_sync();
                arrive_w(&bar.g_free);
                if (krow) {
                    arrive_w(&bar.a_ready[cc & 1]);
                } else {
                    fence_async_smem();
                    arrive_w(&bar.p_ready[cc % kPRing]);
                }
            }
        }
    } else {
        // ------------------------------------------------------------ chain
        set_regs<kChainRegs>();
        // (the state takes half of the registers: a chain's place in memory is looked up
        // where it is used, from the work ring, so that nothing of it stays live)
        const int q4 = warp & 3, wq = warp >> 2, e = 32 * q4 + lane;   // key rows SR wq .., tokens 16 wq ..
        const uint32_t lb = tm + ((uint32_t)(32 * q4) << 16);
        int cc = 0;
        // two bf16 terms of 8 values to TMEM columns hi, lo
        auto put_split = [&](uint32_t hi_at, uint32_t lo_at, const float *x) {
            float hi[4], lo[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) split2(x[2 * m], x[2 * m + 1], hi[m], lo[m]);
            tmem_st4(hi_at, hi);
            tmem_st4(lo_at, lo);
        };
        for (int k = 0; alive; ++k) {
            const int slot = k % kWorks;
            if (!wait_w(&bar.work_full[slot], (k / kWorks) & 1)) { alive = false; break; }
            const volatile Chain *w = &works[slot];
            if (w->n < 0) break;
            // this thread's part of block `at` of `base` (blocks [Hv, Dk, columns]), or NULL
            auto part = [&](const float *base, int64_t at, int64_t extent, DbgSite site) -> float * {
                const int col = 128 * w->tile + e, cols = w->mode == kTransition ? DK : p.Dv;
                if (!base || at < 0 || col >= cols || !dbg_in(at, extent, site)) return nullptr;
                return const_cast<float *>(base) + ((at * p.Hv + w->h) * DK + SR * wq) * cols + col;
            };
            const int nch = w->nch;
            float S[SR];
            {
                const bool first = w->seg == 0;
                const float *src = w->mode != kReal ? nullptr
                                   : first ? part(p.io.init, p.io.init ? pool_slot(p.io.init_slots, w->n, p.io.pool) : -1, p.bd.states, kDbgState)
                                           : part(p.segs.carry, (int64_t)(w->seg - 1) * p.N + w->n, INT64_MAX, kDbgState);
#pragma unroll
                for (int j = 0; j < SR; ++j) S[j] = src ? src[(int64_t)j * p.Dv] : 0.f;
                if (w->mode == kTransition) {
#pragma unroll
                    for (int j = 0; j < SR; ++j) S[j] = SR * wq + j == e ? 1.f : 0.f;
                }
            }
            // the state behind chunk cc - 1, not a number in columns where a value was none
            auto store = [&](float *dst, int cc) {
                const int cols = w->mode == kTransition ? DK : p.Dv;
                if (nch > 0 && (vbad[(cc - 1) % kVRing][q4] >> lane & 1)) {
#pragma unroll 1
                    for (int j = 0; j < SR; ++j, dst += cols) *dst = NAN;
                    return;
                }
#pragma unroll
                for (int j = 0; j < SR; ++j, dst += cols) *dst = S[j];
            };
            __syncwarp();
            bool due = true;   // chunk cc's operand T diag(beta) still to be written
            // T diag(beta) of chunk cc as two bf16 terms: a thread takes 4 columns and rows
            // i, i + 32 as far as they reach the diagonal's 16 x 16 block (what is above the
            // diagonal inside that is zero)
            auto operand = [&](int cc) {
                const float *A = reinterpret_cast<const float *>(sm + SM_A + (cc & 1) * kABytes);
                const int c0 = 4 * (tid & 15), i0 = tid >> 4;
                const float4 be = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm + SM_GATE) +
                                                                    (cc % kGRing) * kGateFloats + c0);
#pragma unroll
                for (int i = i0; i < kC; i += 32)
                    if (i >= (c0 & 48)) {
                        const float4 x = *reinterpret_cast<const float4 *>(A + i * kAP + c0);
                        float b[4] = {x.x, x.y, x.z, x.w}, hi[2], lo[2];
                        mul2(b, be.x, be.y);
                        mul2(b + 2, be.z, be.w);
                        split2(b[0], b[1], hi[0], lo[0]);
                        split2(b[2], b[3], hi[1], lo[1]);
                        uint8_t *dst = sm + SM_T + i * 128 + ((c0 / 8) ^ (i & 7)) * 16 + (c0 & 4) * 2;
                        *reinterpret_cast<float2 *>(dst) = make_float2(hi[0], hi[1]);
                        *reinterpret_cast<float2 *>(dst + kTile) = make_float2(lo[0], lo[1]);
                    }
                fence_async_smem();
                arrive_w(&bar.t_ready);
                arrive_w(&bar.a_free[cc & 1]);
            };
            for (int c = 0;; ++c, ++cc) {
                const uint32_t ph = cc & 1;
                const int i0 = 16 * wq;
                if (c > 0) {
                    // the previous chunk's update D = K^T U
                    if (!wait_w(&bar.d_full, ph ^ 1)) { alive = false; break; }
                    fence_after_sync();
                    const float ec = reinterpret_cast<const float *>(sm + SM_GATE)[((cc - 1) % kGRing) * kGateFloats + 4 * kC];
#pragma unroll
                    for (int j = 0; j < SR; j += 16) {
                        float x[16];
                        tmem_ld16(lb + TM_S + SR * wq + j, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int m = 0; m < 16; m += 2) {
                            const float2 y = __ffma2_rn(make_float2(ec, ec), make_float2(S[j + m], S[j + m + 1]),
                                                        make_float2(x[m], x[m + 1]));
                            S[j + m] = y.x;
                            S[j + m + 1] = y.y;
                        }
                    }
                    const int done = (w->seg * p.segs.G + c) * kC;
                    if (p.io.stride > 0 && done % p.io.stride == 0 && c * kC <= w->len && w->mode == kReal) {
                        const int64_t jc = (int64_t)w->ckpt + done / p.io.stride - 1;
                        if (float *dst = part(p.io.ckpts, jc < p.io.capacity ? pool_slot(p.io.ckpt_slots, jc, p.io.pool) : -1,
                                              p.bd.ckpts, kDbgCkpt))
                            store(dst, cc);
                        __syncwarp();
                    }
                }
                if (c < nch) {
                    // S^T as two bf16 terms
#pragma unroll
                    for (int j = 0; j < SR; j += 8)
                        put_split(lb + TM_S + SR * wq + j / 2, lb + TM_S + SR * wq + SR / 2 + j / 2, S + j);
                    tmem_st_wait();
                    fence_before_sync();
                    arrive_w(&bar.s_ready);
                }
                if (c == nch) break;
                if (due) {   // while K S runs (the products that read the operand of the chunk before are done)
                    if (!wait_w(&bar.i_ready[ph], (cc >> 1) & 1)) { alive = false; break; }
                    operand(cc);
                }
                // (its factors were written before A, from which T came)
                const float *gate = reinterpret_cast<const float *>(sm + SM_GATE) + (cc % kGRing) * kGateFloats + i0;
                if (!wait_w(&bar.x_full, ph)) { alive = false; break; }
                fence_after_sync();
                {   // -e^b rk (K S)^T as two bf16 terms, over itself
                    float x[16];
                    tmem_ld16(lb + TM_X + i0, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int m = 0; m < 16; m += 8) {
#pragma unroll
                        for (int q = m; q < m + 8; q += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(gate + kC + q);
                            mul2(x + q, -f.x, -f.y);
                            mul2(x + q + 2, -f.z, -f.w);
                        }
                        put_split(lb + TM_X + i0 + m / 2, lb + TM_X + i0 + 8 + m / 2, x + m);
                    }
                }
                tmem_st_wait();
                fence_before_sync();
                arrive_w(&bar.r_ready);
                if (!wait_w(&bar.u_full, ph)) { alive = false; break; }
                fence_after_sync();
                {   // U^T for the outputs (over X), and scaled by rk e^(b_C - b) for the state
                    // (over itself), two bf16 terms each
                    float x[16];
                    tmem_ld16(lb + TM_U + i0, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int m = 0; m < 16; m += 8) {
                        put_split(lb + TM_X + i0 + m / 2, lb + TM_X + i0 + 8 + m / 2, x + m);
#pragma unroll
                        for (int q = m; q < m + 8; q += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(gate + 2 * kC + q);
                            mul2(x + q, f.x, f.y);
                            mul2(x + q + 2, f.z, f.w);
                        }
                        put_split(lb + TM_U + i0 + m / 2, lb + TM_U + i0 + 8 + m / 2, x + m);
                    }
                }
                tmem_st_wait();
                fence_before_sync();
                arrive_w(&bar.u_ready);
                // while D runs: the next chunk's operand, if its inverse is there
                due = true;
                if (c + 1 < nch && __all_sync(0xffffffffu, mbar_test(&bar.i_ready[ph ^ 1], ((cc + 1) >> 1) & 1))) {
                    operand(cc + 1);
                    due = false;
                }
            }
            if (alive) {
                const int64_t at = (int64_t)w->seg * p.N + w->n;   // (of segment seg + 1's start; offsets and transitions begin with segment 1)
                float *dst = w->mode == kOffset       ? part(p.segs.offs, at - p.N, INT64_MAX, kDbgState)
                             : w->mode == kTransition ? part(p.segs.trans, at - p.N, INT64_MAX, kDbgState)
                             : !w->last               ? (p.pass == 1 ? part(p.segs.carry, at, INT64_MAX, kDbgState) : nullptr)
                             : part(p.io.fin, p.io.fin ? pool_slot(p.io.final_slots, w->n, p.io.pool) : -1, p.bd.states, kDbgState);
                if (dst) store(dst, cc);
            }
            arrive_w(&bar.work_empty[slot]);
        }
    }
    // (a role that gives up starves the others, which give up in turn)
    if (!alive) record_status(p.st, (int32_t)KDA_ERR_TIMEOUT);
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 0) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------- join
// The states that the segments start from, one after another: segment p + 1
// starts from M_p S_p + B_p (transition and offset of segment p).  A CTA takes 8
// value columns of one (sequence, value head), a thread one row and 4 of them;
// the next M arrives in shared memory while this one is used.
constexpr int kJoinCols = 8;
template <int DK>
__global__ void __launch_bounds__(2 * DK)
gdn_join_kernel(GdnSegs segs, GdnTable tab, int N, int Hv, int Dv)
{
    constexpr int MP = DK + 4;   // row pitch (conflict-free 16-byte reads by rows)
    extern __shared__ __align__(16) float sm[];
    __shared__ __align__(16) float S[2][DK][kJoinCols];
    const int tiles = Dv / kJoinCols, tid = threadIdx.x;
    const int n = (int)(blockIdx.x / ((int64_t)Hv * tiles)), h = (int)(blockIdx.x / tiles % Hv), c0 = (int)(blockIdx.x % tiles) * kJoinCols;
    const int nch = (tab.cu[n + 1] - tab.cu[n] + kC - 1) / kC;
    const int np = min(segs.P, (nch + segs.G - 1) / segs.G);   // segments of this sequence
    const int i = tid % DK, j = 4 * (tid / DK);
    auto block = [&](float *base, int p, int cols) { return base + (((int64_t)p * N + n) * Hv + h) * DK * cols; };
    auto fetch = [&](int p, int buf) {
        const float *m = block(segs.trans, p - 1, DK);
        for (int u = tid; u < DK * DK / 4; u += 2 * DK) {
            const uint32_t dst = smem_u32(sm + buf * DK * MP + (u / (DK / 4)) * MP + 4 * (u % (DK / 4)));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(m + 4 * u) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (np < 3) return;
    fetch(1, 1);
    *reinterpret_cast<float4 *>(&S[1][i][j]) = *reinterpret_cast<const float4 *>(block(segs.carry, 0, Dv) + (int64_t)i * Dv + c0 + j);
    for (int p = 1; p <= np - 2; ++p) {
        const int buf = p & 1;
        const float4 b = *reinterpret_cast<const float4 *>(block(segs.offs, p - 1, Dv) + (int64_t)i * Dv + c0 + j);
        if (p + 1 <= np - 2) {
            fetch(p + 1, buf ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();   // M_p and S_p are there
        const float *m = sm + buf * DK * MP + i * MP;
        float2 y0 = make_float2(b.x, b.y), y1 = make_float2(b.z, b.w);
#pragma unroll 8
        for (int k = 0; k < DK; k += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(m + k);
            const float af[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 s = *reinterpret_cast<const float4 *>(&S[buf][k + q][j]);
                y0 = __ffma2_rn(make_float2(af[q], af[q]), make_float2(s.x, s.y), y0);
                y1 = __ffma2_rn(make_float2(af[q], af[q]), make_float2(s.z, s.w), y1);
            }
        }
        const float4 y = make_float4(y0.x, y0.y, y1.x, y1.y);
        *reinterpret_cast<float4 *>(&S[buf ^ 1][i][j]) = y;
        *reinterpret_cast<float4 *>(block(segs.carry, p, Dv) + (int64_t)i * Dv + c0 + j) = y;
        __syncthreads();   // M_p is free
    }
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeFn encode_fn()
{
    static std::atomic<void *> cached{nullptr};
    void *f = cached.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        cached.store(f, std::memory_order_release);
    }
    return (EncodeFn)f;
}

// [tokens, heads, dim] bf16, boxes of 64 tokens x 64 elements of one head
bool make_map(CUtensorMap *m, EncodeFn fn, const void *p, int64_t tokens, int heads, int dim)
{
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)heads * dim * 2};
    const cuuint32_t box[3] = {64, 1, kC}, step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int join_smem(int dk) { return 2 * dk * (dk + 4) * (int)sizeof(float); }

cudaError_t attributes()
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        const void *fs[] = {(const void *)gdn_tc_kernel<64>, (const void *)gdn_tc_kernel<128>};
        for (const void *f : fs) {
            // the register split counts on the launch's registers: another build is refused
            cudaFuncAttributes at;
            if ((e = cudaFuncGetAttributes(&at, f)) != cudaSuccess) return e;
            if (at.numRegs != (int)kLaunchRegs) return cudaErrorInvalidKernelImage;
            if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem)) != cudaSuccess) return e;
        }
        if ((e = cudaFuncSetAttribute(gdn_join_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, join_smem(128))) != cudaSuccess ||
            (e = cudaFuncSetAttribute(gdn_join_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, join_smem(64))) != cudaSuccess)
            return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_gdn_tc(const GdnArgs &a)
{
    cudaError_t e = attributes();
    if (e != cudaSuccess) return e;
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    // (debug build: rows that the checks take to be missing read as zeros)
    const int64_t rows = a.bounds.tokens < 1 ? 1 : a.bounds.tokens;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, fn, a.q, rows, a.Hk, a.Dk) || !make_map(&mk, fn, a.k, rows, a.Hk, a.Dk) ||
        !make_map(&mv, fn, a.v, rows, a.Hv, a.Dv))
        return cudaErrorInvalidValue;
    const int tiles = (a.Dv + 127) / 128;
    const int64_t sms = device_sm_count(), heads = (int64_t)a.N * a.Hv;
    auto pass = [&](int which, int64_t chains) {
        const Params p{a.g, a.beta, a.v, (__nv_bfloat16 *)a.out, a.N, a.Hk, a.Hv, a.Dv, tiles, chains, which, a.segs, a.tab, a.io,
                       a.status, a.wait_limit, a.bounds};
        const unsigned grid = (unsigned)(chains < sms ? chains : sms);
        if (a.Dk == 128)
            gdn_tc_kernel<128><<<grid, kThreads, kSmem, a.stream>>>(mq, mk, mv, p);
        else
            gdn_tc_kernel<64><<<grid, kThreads, kSmem, a.stream>>>(mq, mk, mv, p);
        return cudaGetLastError();
    };
    const int64_t P = a.segs.P;
    if (P == 1) return pass(0, heads * tiles);
    if ((e = pass(1, heads * (tiles * (P - 1) + P - 2))) != cudaSuccess) return e;
    const unsigned joins = (unsigned)(heads * (a.Dv / kJoinCols));
    if (a.Dk == 128)
        gdn_join_kernel<128><<<joins, 256, join_smem(128), a.stream>>>(a.segs, a.tab, a.N, a.Hv, a.Dv);
    else
        gdn_join_kernel<64><<<joins, 128, join_smem(64), a.stream>>>(a.segs, a.tab, a.N, a.Hv, a.Dv);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return pass(2, heads * tiles * (P - 1));
}

// A chain is serial, so a call with few of them leaves most SMs idle.  It is then
// cut into P segments: pass 1 runs segment 0 with its outputs and, from zeros and
// from the identity, the segments between the first and the last (their end
// state is affine in their start: M S + B); the join forms every segment's start;
// pass 2 runs segments 1 .. P - 1.  That is up to three times the work, in 2 / P of
// the time as long as pass 1 has an SM for each of its chains, and in 3 / P where it
// takes two rounds.  P is the one with the shortest estimate: in units of a chunk's
// time on the chain (4 us), the rounds of both passes, 4 chunks to fill each, 0.7 for
// a step of the join, 3 for the launches.  One sequence of 32768 tokens, 32 heads: 1228 us
// in five segments (three rounds); three (two rounds) took 8 % longer.
GdnSegs plan_gdn_segs(int64_t N, int64_t Hv, int Dv, int64_t max_len)
{
    const int64_t tiles = (Dv + 127) / 128, sms = device_sm_count(), chunks = (max_len + kC - 1) / kC;
    GdnSegs best{1, 0, nullptr, nullptr, nullptr};
    if (N * Hv * tiles > sms) return best;
    double least = (double)chunks + 4;
    for (int64_t P = 3; P <= 64 && 3 * P <= chunks; ++P) {
        const int64_t G = (chunks + P - 1) / P, first = N * Hv * (tiles * (P - 1) + P - 2), second = N * Hv * tiles * (P - 1);
        const int64_t rounds = (first + sms - 1) / sms + (second + sms - 1) / sms;
        const double t = (double)(rounds * (G + 4)) + 0.7 * (double)(P - 2) + 3;
        if (t < least) {
            least = t;
            best.P = (int)P;
            best.G = (int)G;
        }
    }
    return best;
}

KDA_DBG_TAKE(dbg_take_gdn_tc)

}  // namespace kda
