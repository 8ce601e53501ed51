// attn_tc.cu -- causal attention of prompts on the tensor cores (bf16): packed keys and
// values, or a paged cache (bf16 or e4m3) at whose end the new tokens stand.
//
//   S = Q K^T,  P = 2^(S scale - m),  O += P V,  l += sum P     (scale times log2 e)
//
// The two products bound it (4 D multiply-adds' flops a query row and key), so one
// persistent CTA a SM keeps the tensor core busy and everything else runs beside it.  A CTA
// works on two query tiles of 128 rows at once, two heads that share a key head (or, where
// an odd number of heads does, two blocks of tokens): while the softmax of one tile runs, the
// products of the other do, and each tile of 128 keys loaded serves both.
//
//   8 warps   softmax, four of each tile, a thread a row.  S from TMEM, P back over it as
//             bf16 (rounded once, as the product's operand: outputs 2.2e-3 of their norm off where
//             their own rounding is 1.7e-3; a second term would be a third more tensor work).  P refers
//             to a value that is set 16 (2^16) above the maximum and follows it only when that has grown past
//             it, so O is hardly ever rescaled; at the end O / l is written.  The largest weight of a
//             row is thus 2^-16 to 1: l and O, in fp32, lose nothing of values down to 2^-110, and O
//             is not infinite where a row's output is not (it was for values from 2^112 on, when weights went from 1 to 2^16).
//   1         hands out the items and loads: Q once an item, K and V through a ring (TMA,
//             128-byte swizzle)
//   2         issue the products of a tile each, Q K^T of the next keys right behind P V of
//             these: S may be overwritten as soon as P V has read P, which the pipe's order
//             ensures, and an S that is there says that P V before it is done
//   1         tiles of V with keys that not every row sees: a value there that is not finite
//             would reach the rows whose weight is zero, so it becomes a zero, and the rows
//             that see it get NaN in its column at the end
//   (4        e4m3 cache: codes to bf16 tiles)
//
// What bounds it is the way round of one tile, about 2950 cycles a step of 128 keys: its
// products (1024 alone), the softmax, and the barriers between them; the other tile's run
// beside it.  8192 tokens, 32/8 heads: 342 us, 1.6 PFLOP/s; without any softmax 295, at the
// tensor pipe's full rate 242.  Issuing waits for the pipe, so that one thread for both tiles
// left it idle at each of its own waits (3240 cycles, 403 us).  Slower: two threads a row
// (417 us); no look for the maximum but a test of P's exponents (385); P handed over in
// halves (362 to 405); an eighth or a quarter of the exponentials as a polynomial (348, 354:
// issue slots are short, not the exponential unit).
//
// An item of one step takes 3.3 us at D = 64, 2.6 of them without its loads' and stores' traffic: the
// softmax of the masked diagonal, products and barriers, one after another.  Four items
// known ahead, or O of two items in TMEM and the outputs written behind the next one's softmax,
// changed nothing (48 ragged prompts 59 us).
//
// Items (a block of queries and two heads) are sorted by the number of their keys,
// longest first, and handed out one by one.  Where there are few, those with more keys than an
// SM's share of all are cut along the keys; the parts go to the workspace and are joined.
//
// TMEM: S 0, S 1, O 0, O 1, 128 columns each (O: D); P over the first half of its S.
#include <cuda.h>

#include <atomic>

#include "attn.cuh"
#include "tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kBlock = 128;          // query rows of a tile, keys of a step
constexpr int kWorks = 2;
// Warps: eight of the softmax, then the others.  Registers a thread: what the launch gives,
// dealt out anew to the softmax's two warpgroups and to the others, within the launch's total.
template <bool E8> struct Roles {
    static constexpr int kGroups = E8 ? 4 : 3, kThreads = 128 * kGroups, kRowWarps = 8;
    static constexpr int kLoad = 8, kIssue0 = 9, kGuard = 11, kConvert0 = 12;
    static constexpr int kReaders = kRowWarps + 2 + (E8 ? 4 : 1);   // of the items
    static constexpr int kLaunch = E8 ? 128 : 168, kRow = E8 ? 168 : 208, kSide = 88;
    static_assert(2 * kRow + (kGroups - 2) * kSide <= kGroups * kLaunch, "register split");
};
constexpr float kSlack = 16.f;       // how far above the maximum the reference of P is set

template <int D, bool E8> struct Geo {
    static constexpr uint32_t kTile = kBlock * D * 2;            // bytes of Q, K or V of 128 rows
    static constexpr uint32_t kHalf = kBlock * 128;              // 64 elements of each row
    static constexpr int kStages = E8 ? 4 : D == 128 ? 5 : 8;
    static constexpr int kQ = D == 64 ? 2 : 1;                   // items whose Q is there or on its way
    static constexpr uint32_t SM_KV = kQ * 2 * kTile;
    static constexpr uint32_t kRaw = kBlock * D;                 // e4m3 codes of 128 rows
    static constexpr int kRaws = E8 ? 2 : 0;
    static constexpr uint32_t SM_RAW = SM_KV + kStages * kTile;
    static constexpr uint32_t kSmem = SM_RAW + kRaws * kRaw + 1024;
};
static_assert(Geo<128, true>::kSmem <= 227 * 1024 - 2048 && Geo<128, false>::kSmem <= 227 * 1024 - 2048, "shared memory");

// An item as the roles see it; n < 0: no more.
struct Work {
    int n, hk, slot;         // slot: of a part of the keys, -1: all of them
    int h[2], t[2], rows[2]; // head, first row of q and rows of each tile
    int lim[2];              // last key of the tile's first row
    int kt0, kt1, total;     // steps of 128 keys; keys of the sequence
};

struct Barriers {
    uint64_t work_full[kWorks], work_empty[kWorks];
    uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8];
    uint64_t raw_full[8], raw_empty[4];    // V before the guard has seen it (by stage of K and V), or codes
    uint64_t s_full[2], p_ready[2], o_full[2], o_free[2], drain[2];
};

struct Params {
    __nv_bfloat16 *out;
    float *lse;
    PagedKV kv;
    const int32_t *cu, *count;
    int32_t *next;
    const AttnItem *items;
    float *parts;
    float2 *ml;
    int Hq, Hkv, G, pairs, two_heads, last_z;
    float scale;
    int32_t *status;
    uint32_t limit;
    int64_t tokens;
};

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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t by)
{
    uint32_t r;
    asm("mul.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(by));
    return r;
}
// Two e4m3 codes, in the upper bytes of x's halves, times 2^-120 `by` as bf16 values: moved
// to their places, sign, exponent and mantissa give the value times 2^-120.
__device__ __forceinline__ uint32_t e4m3_bf16x2(uint32_t x, uint32_t by)
{
    return mul_bf16x2((x & 0x80008000u) | ((x >> 4) & 0x07F007F0u), by);
}

template <int D, bool E8>
__global__ void __launch_bounds__(Roles<E8>::kThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const Params p)
{
    using GE = Geo<D, E8>;
    using RO = Roles<E8>;
    constexpr int ST = GE::kStages, RS = E8 ? GE::kRaws : 1, QN = GE::kQ;
    constexpr uint32_t TM_S = 0, TM_O = 256;
    extern __shared__ uint8_t raw_sm[];
    __shared__ Barriers bar;
    __shared__ Work works[kWorks];
    __shared__ int first_bad[kWorks][D];        // first key of a guarded step with a value that is not finite
    __shared__ int any_bad[kWorks];
    __shared__ uint32_t tmem_sh;
    uint8_t *sm = raw_sm + ((1024u - (smem_u32(raw_sm) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kWorks; ++i) {
            mbar_init(&bar.work_full[i], 1);
            mbar_init(&bar.work_empty[i], RO::kReaders);
        }
        for (int i = 0; i < ST; ++i) {
            mbar_init(&bar.kv_full[i], E8 ? 4 : 1);
            mbar_init(&bar.kv_empty[i], 2);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&bar.raw_full[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&bar.raw_empty[i], 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.drain[i], 1);
            mbar_init(&bar.p_ready[i], 4);
            mbar_init(&bar.o_full[i], 1);
            mbar_init(&bar.o_free[i], 4);
        }
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_sh, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = tmem_sh;
    next_may_start();
    after_previous();

    bool alive = true;
    auto wait_w = [&](uint64_t *b, uint32_t parity) -> bool {   // whole warps: the same answer in every lane
        return __all_sync(0xffffffffu, wait_limited(b, parity, p.limit));
    };
    auto arrive_w = [&](uint64_t *b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(b);
    };
    // the k-th item of this CTA; the reader releases it
    auto get_work = [&](int k, Work &w) -> bool {
        if (!wait_w(&bar.work_full[k % kWorks], (k / kWorks) & 1)) return false;
        w = works[k % kWorks];
        return true;
    };
    auto guarded = [](const Work &w, int j) -> bool { return (j + 1) * kBlock - 1 > w.lim[0]; };

    if (warp >= RO::kRowWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Roles<E8>::kSide));
        Work w;
        if (warp == RO::kLoad) {
            // ------------------------------------------------------------ items and loads
            const int64_t all = (int64_t)*p.count * p.pairs;
            auto next_id = [&]() -> int {
                int id = 0;
                if (lane == 0) id = atomicAdd(p.next, 1);
                return __shfl_sync(0xffffffffu, id, 0);
            };
            auto item = [&](int id) -> Work {
                Work x;
                x.n = -1;
                if (id >= all) return x;
                const AttnItem it = p.items[id / p.pairs];
                const int pair = id % p.pairs, t0 = p.cu[it.n], len = p.cu[it.n + 1] - t0;
                bool bad;
                x.n = it.n;
                x.total = p.kv.table ? kv_length(p.kv, it.n, &bad) : len;
                x.kt0 = it.kt0;
                x.kt1 = it.kt1;
                x.slot = it.slot < 0 ? -1 : it.slot * p.pairs + pair;
                const int past = x.total - len;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int at = (p.two_heads ? it.block : 2 * it.block + s) * kBlock, left = len - at;
                    x.h[s] = p.two_heads ? 2 * pair + s : pair;
                    x.t[s] = t0 + at;
                    x.rows[s] = left < 0 ? 0 : left > kBlock ? kBlock : left;
                    x.lim[s] = past + at;
                }
                x.hk = x.h[0] / p.G;
                return x;
            };
            // copies into the ring; uses of each raw_full, modulo 2; stages whose last copy reports there
            uint32_t asked = 0, raw = 0, on_raw = 0;
            int q_asked = 0;                     // items whose Q was asked for
            const int rows = p.kv.table ? min(p.kv.page, kBlock) : kBlock, boxes = kBlock / rows;
            Work follow = item(next_id());
            for (int k = 0; alive; ++k) {
                const int slot = k % kWorks;
                w = follow;
                if (k >= kWorks && !(alive = wait_w(&bar.work_empty[slot], (k / kWorks - 1) & 1))) break;
                for (int i = lane; i < D; i += 32) first_bad[slot][i] = INT32_MAX;
                if (lane == 0) {
                    any_bad[slot] = 0;
                    works[slot] = w;
                }
                arrive_w(&bar.work_full[slot]);
                if (w.n < 0) break;
                const int qs = k % QN;
                if (k >= QN && !(alive = wait_w(&bar.q_empty[qs], (k / QN - 1) & 1))) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&bar.q_full[qs], 2 * GE::kTile);
                    for (int s = 0; s < 2; ++s)
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_3d(sm + (2 * qs + s) * GE::kTile + x * GE::kHalf, &mq, 64 * x, w.h[s], w.t[s], &bar.q_full[qs]);
                }
                __syncwarp();
                q_asked = k + 1;
                auto page_z = [&](int j) -> int {          // the lane's box of step j
                    const int at = j * kBlock + lane * rows;
                    if (lane >= boxes || at >= w.total) return p.last_z;
                    const int64_t g = page_of(p.kv, w.n, at);
                    if (g < 0) {
                        if (p.status) atomicCAS(p.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
                        return p.last_z;
                    }
                    return (int)g * p.Hkv + w.hk;
                };
                int z = p.kv.table ? page_z(w.kt0) : 0;
                for (int j = w.kt0; j < w.kt1 && alive; ++j) {
                    const int z_now = z;
                    if (p.kv.table && j + 1 < w.kt1) z = page_z(j + 1);
#pragma unroll
                    for (int which = 0; which < 2; ++which) {
                        constexpr uint32_t RING = E8 ? RS : ST;
                        const uint32_t st = asked % RING;
                        if (asked >= RING && !(alive = wait_w(E8 ? &bar.raw_empty[st] : &bar.kv_empty[st], (asked / RING - 1) & 1))) break;
                        const bool guard = !E8 && which == 1 && guarded(w, j);
                        uint64_t *full = guard || E8 ? &bar.raw_full[st] : &bar.kv_full[st];
                        raw ^= (uint32_t)guard << st;
                        on_raw = (on_raw & ~(1u << st)) | (uint32_t)guard << st;
                        uint8_t *dst = E8 ? sm + GE::SM_RAW + st * GE::kRaw : sm + GE::SM_KV + st * GE::kTile;
                        const CUtensorMap *m = which ? &mv : &mk;
                        const bool one = elect_one();
                        if (one) mbar_arrive_expect_tx(full, E8 ? GE::kRaw : GE::kTile);
                        if (E8) {
                            for (int b = 0; b < boxes; ++b) {
                                const int zb = __shfl_sync(0xffffffffu, z_now, b), y = (j * kBlock + b * rows) & (p.kv.page - 1);
                                if (one) tma_load_3d(dst + b * rows * D, m, 0, y, zb, full);
                            }
                        } else if (!p.kv.table) {
                            // (the sequence's first row of k and v is that of its first query)
                            if (one)
                                for (int x = 0; x < D / 64; ++x)
                                    tma_load_3d(dst + x * GE::kHalf, m, 64 * x, w.hk, w.t[0] - w.lim[0] + j * kBlock, full);
                        } else {
                            for (int b = 0; b < boxes; ++b) {
                                const int zb = __shfl_sync(0xffffffffu, z_now, b), y = (j * kBlock + b * rows) & (p.kv.page - 1);
                                if (one)
                                    for (int x = 0; x < D / 64; ++x)
                                        tma_load_3d(dst + x * GE::kHalf + b * rows * 128, m, 64 * x, y, zb, full);
                            }
                        }
                        __syncwarp();
                        ++asked;
                    }
                    // the next item, once and early: its reads take longer than a step
                    if (alive && (j == w.kt0 + 1 || w.kt1 - w.kt0 == 1)) follow = item(next_id());
                }
            }
            if (!alive) {   // (else the issuer has waited for all of them) no copy outlives the CTA
                for (int i = 0; i < QN; ++i)
                    if (q_asked > i) mbar_wait_bounded(&bar.q_full[i], ((q_asked - 1 - i) / QN) & 1, kDrainLimit);
                constexpr uint32_t RING = E8 ? RS : ST;
                for (uint32_t i = 0; i < RING; ++i)
                    if (asked > i) {
                        const uint32_t uses = (asked - 1 - i) / RING + 1;
                        if (E8) mbar_wait_bounded(&bar.raw_full[i], (uses - 1) & 1, kDrainLimit);
                        else if (on_raw >> i & 1) mbar_wait_bounded(&bar.raw_full[i], ~(raw >> i) & 1, kDrainLimit);
                        else mbar_wait_bounded(&bar.kv_full[i], (uses - 1) & 1, kDrainLimit);
                    }
            }
        } else if (warp == RO::kIssue0 || warp == RO::kIssue0 + 1) {
            // ------------------------------------------------------------ products of tile s, by one thread
            const int s = warp - RO::kIssue0;
            if (elect_one()) {
                constexpr uint32_t id_s = idesc_bf16(128, 128), id_o = idesc_bf16(128, D) | kIdescBMn;
                uint32_t used = 0, ready = 0;
                auto wait = [&](uint64_t *b, uint32_t parity) { return alive = wait_limited(b, parity, p.limit); };
                auto scores = [&](uint32_t st, int qs) {
                    const uint32_t a = sb + (2 * qs + s) * GE::kTile, b = sb + GE::SM_KV + st * GE::kTile;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t at = (i >> 2) * GE::kHalf + (i & 3) * 32;
                        mma_f16(tm + TM_S + 128 * s, make_desc_sw128(a + at, 0), make_desc_sw128(b + at, 0), id_s, i > 0);
                    }
                    mma_commit(&bar.s_full[s]);
                    mma_commit(&bar.kv_empty[st]);
                };
                for (int k = 0; alive; ++k) {
                    if (!wait(&bar.work_full[k % kWorks], (k / kWorks) & 1)) break;
                    const int n = works[k % kWorks].n, kt0 = works[k % kWorks].kt0, kt1 = works[k % kWorks].kt1;
                    mbar_arrive(&bar.work_empty[k % kWorks]);
                    if (n < 0) break;
                    const int qs = k % QN;
                    if (!wait(&bar.q_full[qs], (k / QN) & 1) || !wait(&bar.kv_full[used % ST], (used / ST) & 1)) break;
                    fence_after_sync();
                    scores(used % ST, qs);
                    if (kt1 - kt0 == 1) mma_commit(&bar.q_empty[qs]);
                    ++used;
                    for (int j = kt0; j < kt1; ++j) {
                        const uint32_t vs = used % ST, ks = (used + 1) % ST;
                        const bool more = j + 1 < kt1;
                        // (everything that may have to be waited for before the first product: the pipe runs dry
                        // soon after the last was issued)
                        if (!wait(&bar.kv_full[vs], (used / ST) & 1)) break;
                        if (more && !wait(&bar.kv_full[ks], ((used + 1) / ST) & 1)) break;
                        if (j == kt0 && k > 0 && !wait(&bar.o_free[s], (k - 1) & 1)) break;
                        if (!wait(&bar.p_ready[s], ready++ & 1)) break;
                        fence_after_sync();
                        const uint32_t b = sb + GE::SM_KV + vs * GE::kTile;
#pragma unroll
                        for (int i = 0; i < kBlock / 16; ++i)
                            mma_f16_ts(tm + TM_O + D * s, tm + TM_S + 128 * s + 8 * i, make_desc_sw128(b + i * 2048, GE::kHalf), id_o,
                                       j > kt0 || i > 0);
                        mma_commit(&bar.kv_empty[vs]);
                        if (more) {
                            scores(ks, qs);
                            if (j + 2 == kt1) mma_commit(&bar.q_empty[qs]);
                        } else {
                            mma_commit(&bar.o_full[s]);
                        }
                        used += more ? 2 : 1;
                    }
                }
                mma_commit(&bar.drain[s]);   // no product outlives the CTA
                mbar_wait_bounded(&bar.drain[s], 0, kDrainLimit);
            }
            __syncwarp();
            alive = __all_sync(0xffffffffu, alive);
        } else if (E8 && warp >= RO::kConvert0) {
            // ------------------------------------------------------------ codes to bf16
            // (values of keys behind the sequence's end are zeros; so are those of rows whose scale
            // is not finite, in steps with keys that not every row sees: see the guard)
            uint32_t it = 0;
            const int r0 = (warp - RO::kConvert0) * 32;
            constexpr int RP = 256 / D, NI = 32 / RP;      // rows at once, times
            const int r = lane / (D / 8), c = lane % (D / 8);
            for (int k = 0; alive; ++k) {
                const int slot = k % kWorks;
                if (!(alive = get_work(k, w))) break;
                if (w.n < 0) {
                    arrive_w(&bar.work_empty[slot]);
                    break;
                }
                auto row_of = [&](int j) -> int64_t {      // of the cache's scales, this lane's row of step j
                    const int key = j * kBlock + r0 + lane;
                    if (j >= w.kt1 || key >= w.total) return -1;
                    const int64_t g = page_of(p.kv, w.n, key);
                    return g < 0 ? -1 : (g * p.Hkv + w.hk) * p.kv.page + (key & (p.kv.page - 1));
                };
                // rows two steps ahead, scales one
                int64_t ahead = row_of(w.kt0);
                float sk = ahead < 0 ? 0.f : p.kv.ks[ahead], sv = ahead < 0 ? 0.f : p.kv.vs[ahead];
                ahead = row_of(w.kt0 + 1);
                for (int j = w.kt0; j < w.kt1 && alive; ++j) {
                    const float k_now = sk, v_now = sv;
                    sk = ahead < 0 ? 0.f : p.kv.ks[ahead];
                    sv = ahead < 0 ? 0.f : p.kv.vs[ahead];
                    ahead = row_of(j + 2);
#pragma unroll
                    for (int which = 0; which < 2; ++which, ++it) {
                        const uint32_t rs = it % RS, st = it % ST;
                        if (!(alive = wait_w(&bar.raw_full[rs], (it / RS) & 1))) break;
                        if (it >= ST && !(alive = wait_w(&bar.kv_empty[st], (it / ST - 1) & 1))) break;
                        float sc = which ? v_now : k_now;
                        if (which && guarded(w, j) && !(fabsf(sc) < __int_as_float(0x7f800000))) {
#pragma unroll 1
                            for (int d = 0; d < D; ++d) atomicMin(&first_bad[slot][d], j * kBlock + r0 + lane);
                            any_bad[slot] = 1;
                            sc = 0.f;
                        }
                        // 2^120 sc, in two factors where one would be beyond bf16
                        const bool large = __any_sync(0xffffffffu, sc > 128.f);
                        const float f1 = large ? 0x1p120f : sc * 0x1p120f;
                        const uint32_t s1 = pack_bf16(f1, f1), s2 = pack_bf16(sc, sc);
                        // 8 codes a lane, D / 8 lanes a row: one 16-byte piece of bf16 each, so that the
                        // eight lanes that store at once meet no bank twice
                        const uint8_t *src = sm + GE::SM_RAW + rs * GE::kRaw + r0 * D + lane * 8;
                        uint8_t *dst = sm + GE::SM_KV + st * GE::kTile + (c >> 3) * GE::kHalf + (r0 + r) * 128;
#pragma unroll
                        for (int i0 = 0; i0 < NI; i0 += 8) {       // (no load moves ahead of a store by itself)
                            uint2 x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const uint2 *>(src + (i0 + i) * 256);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int row = (i0 + i) * RP + r;     // (r0 is a multiple of 8)
                                const uint32_t f = __shfl_sync(0xffffffffu, s1, row);
                                *reinterpret_cast<uint4 *>(dst + (i0 + i) * RP * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                                    make_uint4(e4m3_bf16x2(__byte_perm(x[i].x, 0, 0x1100), f), e4m3_bf16x2(__byte_perm(x[i].x, 0, 0x3322), f),
                                               e4m3_bf16x2(__byte_perm(x[i].y, 0, 0x1100), f), e4m3_bf16x2(__byte_perm(x[i].y, 0, 0x3322), f));
                            }
                        }
                        if (large)
#pragma unroll 1
                            for (int i = 0; i < NI; ++i) {
                                const int row = i * RP + r;
                                const uint32_t f = __shfl_sync(0xffffffffu, s2, row);
                                uint4 &y = *reinterpret_cast<uint4 *>(dst + i * RP * 128 + (((c & 7) ^ (row & 7)) << 4));
                                y = make_uint4(mul_bf16x2(y.x, f), mul_bf16x2(y.y, f), mul_bf16x2(y.z, f), mul_bf16x2(y.w, f));
                            }
                        fence_async_smem();
                        arrive_w(&bar.raw_empty[rs]);
                        arrive_w(&bar.kv_full[st]);
                    }
                }
                arrive_w(&bar.work_empty[slot]);
            }
        } else if (!E8 && warp == RO::kGuard) {
            // ------------------------------------------------------------ guard
            uint32_t used = 0, phase = 0;
            for (int k = 0; alive; ++k) {
                const int slot = k % kWorks;
                if (!(alive = get_work(k, w))) break;
                if (w.n < 0) {
                    arrive_w(&bar.work_empty[slot]);
                    break;
                }
                for (int j = w.kt0; j < w.kt1 && alive; ++j) {
                    const uint32_t st = (used + 1) % ST;   // K, then V
                    used += 2;
                    if (!guarded(w, j)) continue;
                    if (!(alive = wait_w(&bar.raw_full[st], phase >> st & 1))) break;
                    phase ^= 1u << st;
                    uint8_t *v = sm + GE::SM_KV + st * GE::kTile;
                    uint32_t odd = 0;
#pragma unroll 8
                    for (int i = lane; i < (int)GE::kTile / 16; i += 32) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(v + i * 16);
                        // an exponent of all ones carries into the bit above
                        odd |= ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) |
                               ((x.z & 0x7F807F80u) + 0x00800080u) | ((x.w & 0x7F807F80u) + 0x00800080u);
                    }
                    if (__any_sync(0xffffffffu, odd & 0x80008000u)) {
                        for (int i = lane; i < (int)GE::kTile / 2; i += 32) {
                            uint16_t *at = reinterpret_cast<uint16_t *>(v) + i;
                            if ((*at & 0x7F80) != 0x7F80) continue;
                            *at = 0;
                            // row, 16-byte piece (swizzled) and element of the byte offset 2 i
                            const int half = 2 * i / (int)GE::kHalf, in = 2 * i % (int)GE::kHalf, r = in >> 7;
                            const int d = 64 * half + ((((in >> 4) & 7) ^ (r & 7)) << 3) + ((in & 15) >> 1), key = j * kBlock + r;
                            if (key < w.total) {
                                atomicMin(&first_bad[slot][d], key);
                                any_bad[slot] = 1;
                            }
                        }
                    }
                    fence_async_smem();
                    arrive_w(&bar.kv_full[st]);
                }
                arrive_w(&bar.work_empty[slot]);
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Roles<E8>::kRow));
        const int s = warp >> 2, row = tid & 127;
        const uint32_t at = tm + ((uint32_t)(warp & 3) << 21);   // lanes 32 (warp & 3) ..
        const uint32_t ts = at + TM_S + 128 * s, to = at + TM_O + D * s;
        uint32_t seen = 0;
        for (int k = 0; alive; ++k) {
            const int slot = k % kWorks;
            const Work &w = works[slot];         // (in shared memory until this warp releases it)
            if (!(alive = wait_w(&bar.work_full[slot], (k / kWorks) & 1))) break;
            if (w.n < 0) {
                arrive_w(&bar.work_empty[slot]);
                break;
            }
            const int lim = w.lim[s] + row, kt0 = w.kt0, kt1 = w.kt1;   // lim: last key of this row
            float mref = -INFINITY, l = 0.f;
            for (int j = kt0; j < kt1; ++j) {
                if (!(alive = wait_w(&bar.s_full[s], seen++ & 1))) break;
                fence_after_sync();
                float x[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, x[i]);
                tmem_ld_wait();
                const int n = lim - j * kBlock;          // last column that the row sees
                if (__any_sync(0xffffffffu, n < kBlock - 1)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (32 * i + c > n) x[i][c] = -INFINITY;
                }
                float top[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    top[i] = x[i][0];
#pragma unroll
                    for (int c = 1; c < 32; ++c) top[i] = fmaxf(top[i], x[i][c]);
                }
                const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale;
                const bool up = t > mref;
                if (__any_sync(0xffffffffu, up)) {
                    const float f = up ? exp2f(mref - (t + kSlack)) : 1.f;   // (0 where mref was -inf)
                    if (up) mref = t + kSlack;
                    l *= f;
                    if (j > kt0) {                       // S is there, so P V of the steps before is done
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
                            float o[16];
                            tmem_ld16(to + 16 * i, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] *= f;
                            tmem_st16(to + 16 * i, o);
                        }
                    }
                }
                const float m = mref == -INFINITY ? 0.f : mref;
                const float2 sc = make_float2(p.scale, p.scale), mm = make_float2(-m, -m);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y[16];                         // P, two to a word
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float2 e = __ffma2_rn(make_float2(x[i][c], x[i][c + 1]), sc, mm);
                        const float2 q = make_float2(ex2_ftz(e.x), ex2_ftz(e.y));
                        sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], q);
                        y[c >> 1] = __uint_as_float(pack_bf16(q.x, q.y));
                    }
                    tmem_st16(ts + 16 * i, y);
                }
                tmem_st_wait();
                fence_before_sync();
                arrive_w(&bar.p_ready[s]);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (!alive) break;
            if (!(alive = wait_w(&bar.o_full[s], k & 1))) break;
            fence_after_sync();
            const int64_t tok = (int64_t)w.t[s] + row;
            const int head = w.h[s];
            const bool bad = any_bad[slot] != 0;
            const float inv = w.slot >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
            const bool mine = row < w.rows[s] && dbg_in(tok, p.tokens, kDbgTokenRow);
            __nv_bfloat16 *dst = p.out + (tok * p.Hq + head) * D;
            float *part = p.parts + (((int64_t)w.slot * 2 + s) * kBlock + row) * D;
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
                float o[16];
                tmem_ld16(to + 16 * i, o);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    o[c] *= inv;
                    if (bad && first_bad[slot][16 * i + c] <= lim) o[c] = __int_as_float(0x7fc00000);
                }
                if (mine) {
                    if (w.slot >= 0) {
#pragma unroll
                        for (int c = 0; c < 16; c += 4)
                            *reinterpret_cast<float4 *>(part + 16 * i + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; c += 8)
                            *reinterpret_cast<uint4 *>(dst + 16 * i + c) = make_uint4(pack_bf16(o[c], o[c + 1]), pack_bf16(o[c + 2], o[c + 3]),
                                                                                      pack_bf16(o[c + 4], o[c + 5]), pack_bf16(o[c + 6], o[c + 7]));
                    }
                }
                __syncwarp();
            }
            fence_before_sync();
            arrive_w(&bar.o_free[s]);
            if (mine) {
                if (w.slot >= 0) p.ml[((int64_t)w.slot * 2 + s) * kBlock + row] = make_float2(mref, l);
                else if (p.lse) p.lse[tok * p.Hq + head] = l == 0.f ? -INFINITY : (mref + log2f(l)) * 0.69314718f;
            }
            arrive_w(&bar.work_empty[slot]);
        }
    }
    if (!alive && lane == 0 && p.status) atomicCAS(p.status, 0, (int32_t)KDA_ERR_TIMEOUT);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 0) tmem_dealloc(tm, 512);
}

// Joins the parts of the items that were cut: a warp a row, parts in order of the keys.
template <int D> __global__ void __launch_bounds__(256) attn_tc_join_kernel(const Params p, const AttnJoin *joins, const int32_t *count)
{
    constexpr int E = D / 32;
    after_previous();
    const int lane = threadIdx.x & 31, d = lane * E;
    const int64_t rows = (int64_t)*count * p.pairs * 2 * kBlock;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < rows; i += (int64_t)gridDim.x * 8) {
        const int row = (int)(i % kBlock), s = (int)(i / kBlock % 2), pair = (int)(i / (2 * kBlock) % p.pairs);
        const AttnJoin jn = joins[i / (2 * kBlock) / p.pairs];
        const int t0 = p.cu[jn.n], len = p.cu[jn.n + 1] - t0, at = (p.two_heads ? jn.block : 2 * jn.block + s) * kBlock + row;
        if (at >= len) continue;
        const int64_t tok = (int64_t)t0 + at;
        if (!dbg_in(tok, p.tokens, kDbgTokenRow)) continue;
        auto part = [&](int j) -> int64_t { return (((int64_t)(jn.slot + j) * p.pairs + pair) * 2 + s) * kBlock + row; };
        // (a lane a part's maximum and sum: all of a row's loads are in flight together)
        float m = -INFINITY, l = 0.f, o[E];
        for (int j0 = 0; j0 < jn.parts; j0 += 32) m = fmaxf(m, j0 + lane < jn.parts ? p.ml[part(j0 + lane)].x : -INFINITY);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int j0 = 0; j0 < jn.parts; j0 += 32) {
            const float2 mine = j0 + lane < jn.parts ? p.ml[part(j0 + lane)] : make_float2(-INFINITY, 0.f);
            const float w = mine.x == -INFINITY ? 0.f : exp2f(mine.x - m), wl = w * mine.y;
            const int n = min(32, jn.parts - j0);
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                const float f = __shfl_sync(0xffffffffu, w, j);
                l += __shfl_sync(0xffffffffu, wl, j);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 x = *reinterpret_cast<const float2 *>(p.parts + part(j0 + j) * D + d + e);
                    o[e] = fmaf(f, x.x, o[e]);
                    o[e + 1] = fmaf(f, x.y, o[e + 1]);
                }
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int h = p.two_heads ? 2 * pair + s : pair;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t *>(p.out + (tok * p.Hq + h) * D + d + e) = pack_bf16(o[e] * inv, o[e + 1] * inv);
        if (p.lse && lane == 0) p.lse[tok * p.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
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

// [z, y, D] with rows y and blocks z so many elements apart: bf16 in boxes of 64 elements, by and
// bz, 128-byte swizzle; bytes (e4m3) in boxes of whole rows as they are
bool make_map(CUtensorMap *m, EncodeFn fn, bool bytes, const void *base, int D, int64_t y, int64_t z, int64_t y_step, int64_t z_step,
              int by, int bz)
{
    const int size = bytes ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)y, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)y_step * size, (cuuint64_t)z_step * size};
    const cuuint32_t box[3] = {(cuuint32_t)(bytes ? D : 64), (cuuint32_t)by, (cuuint32_t)bz}, step[3] = {1, 1, 1};
    return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
              box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E8> cudaError_t attributes_of()
{
    // the register split counts on the launch's registers: another build is refused
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, attn_tc_kernel<D, E8>);
    if (e != cudaSuccess) return e;
    if (at.numRegs != Roles<E8>::kLaunch) return cudaErrorInvalidKernelImage;
    return cudaFuncSetAttribute(attn_tc_kernel<D, E8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo<D, E8>::kSmem);
}

cudaError_t attributes()
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
        if ((e = attributes_of<64, false>()) != cudaSuccess || (e = attributes_of<128, false>()) != cudaSuccess ||
            (e = attributes_of<64, true>()) != cudaSuccess || (e = attributes_of<128, true>()) != cudaSuccess)
            return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

template <int D, bool E8>
cudaError_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const Params &p, unsigned grid, cudaStream_t s)
{
    return launch_following(attn_tc_kernel<D, E8>, dim3(grid), Roles<E8>::kThreads, Geo<D, E8>::kSmem, s, mq, mk, mv, p);
}

}  // namespace

bool attn_on_tc(kda_dtype dtype) { return dtype == KDA_DTYPE_BF16; }

cudaError_t launch_attn_tc(const AttnArgs &a)
{
    cudaError_t e = attributes();
    if (e != cudaSuccess) return e;
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    // (debug build: rows that the checks take to be missing read as zeros)
    const int64_t rows = a.bounds.tokens < 1 ? 1 : a.bounds.tokens, D = a.D;
    const bool paged = a.kv.table != nullptr;
    const int64_t z = paged ? a.kv.pages * a.Hkv : 0;
    if (z >= INT32_MAX) return cudaErrorNotSupported;
    CUtensorMap mq, mk, mv;
    const bool e8 = paged && a.kv_dtype == KDA_DTYPE_E4M3;
    bool ok = make_map(&mq, fn, false, a.q, a.D, a.Hq, rows, D, a.Hq * D, 1, kBlock);
    for (int i = 0; i < 2; ++i) {
        CUtensorMap *m = i ? &mv : &mk;
        const void *base = paged ? (i ? a.kv.v : a.kv.k) : i ? a.v : a.k;
        if (!paged) ok = ok && make_map(m, fn, false, base, a.D, a.Hkv, rows, D, a.Hkv * D, 1, kBlock);
        // (no page at all: everything is out of range)
        else ok = ok && make_map(m, fn, e8, base, a.D, a.kv.page, z ? z : 1, D, a.kv.page * D,
                                 a.kv.page < kBlock ? a.kv.page : kBlock, 1);
    }
    if (!ok) return cudaErrorInvalidValue;
    Params p;
    p.out = (__nv_bfloat16 *)a.out; p.lse = a.lse; p.kv = a.kv; p.cu = a.cu;
    p.count = a.plan.count; p.next = a.plan.next; p.items = a.plan.items; p.parts = a.plan.parts; p.ml = a.plan.ml;
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.two_heads = a.plan.two_heads; p.pairs = a.plan.pairs;
    p.last_z = (int)(z ? z : 1); p.scale = a.scale; p.status = a.status; p.limit = a.wait_limit; p.tokens = a.bounds.tokens;
    const int64_t sms = device_sm_count(), most = a.plan.capacity * p.pairs;
    const unsigned grid = (unsigned)(most < sms ? most : sms);
    e = (a.D == 128 ? e8 ? launch<128, true> : launch<128, false> : e8 ? launch<64, true> : launch<64, false>)(mq, mk, mv, p, grid, a.stream);
    if (e != cudaSuccess || !a.plan.split) return e;
    return launch_following(a.D == 128 ? attn_tc_join_kernel<128> : attn_tc_join_kernel<64>, dim3((unsigned)(2 * sms)), 256, 0, a.stream, p,
                            a.plan.joins, a.plan.join_count);
}

KDA_DBG_TAKE(dbg_take_attn_tc)

}  // namespace kda
