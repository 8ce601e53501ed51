"""The attention layers at the ends of their types' ranges, and the precision of each kernel's own weights, against the
float64 definitions (tests/attn_reference.py)."""
import math

import pytest
import torch

import attn_reference as ref
from attn_reference import EPS16, EPS32, F8, F64, f64
from linear_attention_serving_k1_gb300 import kda
from test_gpu_attn import KV, _check_packed, _packed, _size, i32, word

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
INVALID = kda.STATUS_CODES["KDA_ERR_INVALID_ARG"]
TOP32 = float(torch.finfo(FP32).max)


def bits32(x):
    return float(torch.tensor(x, dtype=torch.int32).view(FP32))


# ---------------------------------------------------------------- the largest fp32 values
# (a first term of 11 bits, rounded to nearest, is infinite from 0x7f7ff000 on)
@pytest.mark.parametrize("big", [0x7F7FFFFF, 0x7F7FF000, 0x7F7FEFFF], ids=["top", "first", "below"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 2), (64, 3, 3), (64, 160, 80)])
def test_fp32_prefill_takes_the_largest_values(D, Hq, Hkv, big):
    """A finite value is its weight times itself in the rows that see it, and nothing in the others."""
    lens, top = [200, 150], bits32(big)
    q, k, v, cu = _packed(lens, Hq, Hkv, D, FP32, 3)
    base, bl = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    v[70, 0, 5], v[130, Hkv - 1, 9], v[199, 0, 0] = top, -top, top
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    assert torch.equal(lse, bl)
    rep = Hq // Hkv
    changed = torch.zeros(out.shape, dtype=torch.bool)
    changed[70:200, :rep, 5] = changed[130:200, -rep:, 9] = changed[199, :rep, 0] = True
    assert torch.equal(out.cpu()[~changed], base.cpu()[~changed])
    if Hq < 10:
        _check_packed(out, lse, q, k, v, lens)
    else:
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("m", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_fp32_over_the_cache_takes_the_largest_values(D, m):
    c = ref.Case([m, m], [200, 60], 4, 2, D, 16, FP32, "same", seed=5)
    k, v, table, lens = c.cache
    q = c.qd.view(2, m, 4, D)
    base, bl = kda.attn_decode_multi(q, *c.cache, want_lse=True)
    j = 200 + m - 1                                 # the last of sequence 0's tokens
    for n, at, h, d, x in ((0, j, 1, 7, TOP32), (1, 13, 0, 2, -TOP32)):
        v[int(table[n, at // 16]), h, at % 16, d] = x
        c.v[n][at, h, d] = x
    out, lse = kda.attn_decode_multi(q, *c.cache, want_lse=True)
    assert torch.equal(lse, bl) and torch.equal(out[0, :m - 1], base[0, :m - 1])
    c.check(out, lse)
    out, lse = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True)
    c.check(out, lse)


@pytest.mark.parametrize("large", ["q", "k"])
def test_fp32_scores_of_the_largest_values(large):
    """The largest value times 2^-126 is a score like any other."""
    lens, D = [90], 64
    q, k, v, cu = _packed(lens, 2, 1, D, FP32, 6)
    small = 2.0 ** -126
    if large == "k":
        q[:, :, 5] = small
        k[40, 0, 5], k[41, 0, 5] = TOP32, -TOP32
    else:
        k[:, :, 5] = small
        q[40:60, 1, 5] = TOP32
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, q, k, v, lens)


# ---------------------------------------------------------------- e4m3 rows that hold no number
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_append_writes_no_code_that_is_not_a_number(D, page):
    """A row with a value that is not finite says so in its scale alone: a product of its codes with a weight of zero stays
    zero, so the earlier ones of several decoded tokens do not see it."""
    m, Hq, Hkv, past = 4, 4, 2, 60
    c = ref.Case([m], [past], Hq, Hkv, D, page, BF16, "e4m3", seed=8)
    k, v, table, lens = c.cache
    q = c.qd.view(1, m, Hq, D)
    g = torch.Generator().manual_seed(21)
    kn, vn = (torch.randn(m, Hkv, D, generator=g).to(BF16) for _ in range(2))
    pos, ids = i32(range(past, past + m)), i32([0] * m)

    def run(kk, vv):
        kda.kv_append(None, kk.cuda(), vv.cuda(), pos, seq_ids=ids, page_table=table, k_cache=k, v_cache=v, **c.scales)
        return [kda.attn_decode_multi(q, *c.cache, **c.scales)[0], kda.attn_prefill_paged(c.qd, *c.cache, c.cu, **c.scales)[0].view(q.shape)]

    base = run(kn, vn)
    for bad in (math.nan, math.inf, -math.inf):
        for which in "kv":
            x = (vn if which == "v" else kn).clone()
            x[2, 1, 9] = bad
            got = run(*((kn, x) if which == "v" else (x, vn)))
            for cache in (k, v):
                assert int(((cache.view(torch.uint8) & 0x7F) == 0x7F).sum()) == 0
            want = torch.zeros(q.shape, dtype=torch.bool)
            want[0, 2:, 2:] = True
            for o, b in zip(got, base):
                assert torch.equal(~torch.isfinite(o).cpu(), want), (bad, which)
                assert torch.equal(o.cpu()[~want], b.cpu()[~want])


# ---------------------------------------------------------------- large values under growing scores
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("jump", [6.0, 10.5])
def test_prefill_large_values_behind_a_growing_maximum(dtype, D, jump):
    """A key whose score is e^jump of the earlier ones', with a value near the largest of the type."""
    L = 300
    g = torch.Generator().manual_seed(31)
    q, k = torch.zeros(L, 2, D), torch.zeros(L, 1, D)
    q[:, :, 0], k[200, 0, 0] = 4.0, jump * D ** 0.5 / 4
    k[:200, 0, 1] = torch.randn(200, generator=g)
    v = torch.randn(L, 1, D, generator=g)
    v[200, 0, 3], v[200, 0, 4], v[5, 0, 6] = 3.0e38, -2.0e38, 3.0e38
    q, k, v = (x.to(dtype) for x in (q, k, v))
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    _check_packed(out, lse, q, k, v, [L])


@pytest.mark.parametrize("dtype,kv", KV)
@pytest.mark.parametrize("past", [250, 3000])
def test_prefill_paged_large_values_behind_a_growing_maximum(dtype, kv, past):
    """The same over a cache (3000: cut along the keys)."""
    m, D, page = 5, 128, 32
    c = ref.Case([m], [past], 2, 1, D, page, dtype, kv, seed=9)
    k, v, table, lens = c.cache
    n = past + m
    c.q[:], c.q[:, :, 0] = 0, 4.0
    c.qd.copy_(c.q)
    rows = torch.zeros(n, 1, D)
    rows[200, 0, 0] = 6.5 * D ** 0.5 / 4
    values = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(32))
    values[200] *= 2.0e38 / values[200].abs().max()
    rows, values = rows.to(dtype).cuda(), values.to(dtype).cuda()
    kda.kv_append(None, rows, values, i32(range(n)), seq_ids=i32([0] * n), page_table=table, k_cache=k, v_cache=v, **c.scales)
    t = table.cpu()
    sk, sv = (None if s is None else s.cpu() for s in c.scales.values())
    if kv == "e4m3":
        c.k, c.v = [c._read(k.cpu(), sk, t[0], n)], [c._read(v.cpu(), sv, t[0], n)]
    else:
        c.k, c.v = [f64(rows)], [f64(values)]
    out, lse = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, **c.scales)
    c.check(out, lse)


@pytest.mark.parametrize("R,inter", [(64, False), (64, True), (24, False)])
def test_append_of_infinities(R, inter):
    """Rotated keys beside an e4m3 cache are infinite or not a number where they are beside a bf16 one."""
    T, D, page = 20, 64, 32
    g = torch.Generator().manual_seed(41)
    k = torch.randn(T, 2, D, generator=g).to(BF16)
    k[3, 0, 5], k[4, 1, 9], k[5, 0, 2], k[5, 0, 2 + R // 2], k[6, 1, 60] = math.inf, -math.inf, math.inf, math.inf, math.inf
    k[7, 0, 3], k[8, 1, 1], k[8, 1, 1 + R // 2] = math.nan, 3.3e38, -3.3e38
    pos = i32([4 * i + 1 for i in range(T)])
    freq, _ = kda.rope_frequencies(R)
    outs = []
    for kv in (BF16, F8):
        cache = [torch.zeros(3, 2, page, D, device="cuda").to(kv) for _ in range(2)]
        sc = {n: torch.zeros(3, 2, page, device="cuda") if kv == F8 else None for n in ("k_scale", "v_scale")}
        outs.append(kda.kv_append(None, k.cuda(), k.cuda(), pos, seq_ids=torch.zeros_like(pos), page_table=i32([[0, 1, 2]]), k_cache=cache[0],
                                  v_cache=cache[1], inv_freq=freq.cuda(), interleaved=inter, want_k=True, **sc)[1].cpu().float())
    a, b = outs
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.isposinf(), b.isposinf()) and torch.equal(a.isneginf(), b.isneginf())
    assert int(a.isinf().sum()) >= 6


# ---------------------------------------------------------------- each decode kernel's own weights
def _sharp(c, out, lse, kv):
    """Outputs of a decode call to what its weights allow, the output's own rounding aside.  bf16: two bf16 terms, half a
    step of the second (2^-8 of 2^-8).  e4m3: f16 weights times the value's scale, referred to a power of two near the largest
    so far: half a step (2^-11 of itself, 2^-25 of the reference where that is more; the reference is at most the largest, the codes
    at most 448), and q as f16 with its row's power of two (elements off by 2^-25 of that)."""
    D = c.q.shape[-1]
    want, wl, A, d = ref.attend_all(f64(c.q), c.k, c.v, c.lens, c.past, D ** -0.5)
    n = max(a + b for a, b in zip(c.lens, c.past))
    ds = (D / 4 + 8) * EPS32 * d
    weight = 2.0 ** -16
    few = torch.zeros_like(A[..., :1])
    if kv == "e4m3":
        weight, t = 2.0 ** -11, 0
        for i, m in enumerate(c.lens):
            rep = c.q.shape[1] // c.k[i].shape[1]
            reach = (c.k[i].abs().sum(-1).amax(0) * D ** -0.5).repeat_interleave(rep)        # sum |k|, the largest of a head
            ds[t:t + m] += 2.0 ** -25 * f64(c.q[t:t + m]).abs().amax(-1) * reach
            s = ref.scale_of(c.v[i]).amax(0).repeat_interleave(rep)                          # (stored values: at most half of it)
            few[t:t + m, :, 0] = 2.0 ** -25 * 448 * len(c.v[i]) * 2 * s / torch.exp(wl[t:t + m] - _top(c, i, t, m))
            t += m
    more = 2 * ds + (4 * math.sqrt(n) + 16) * EPS32
    tol = EPS16 * want.abs() + (1 + EPS16) * ((more[..., None] + weight) * A + few) + 1e-30
    err = (f64(out).reshape(want.shape) - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((f64(lse).reshape(wl.shape) - wl).abs() <= ds + (4 * math.sqrt(n) + 16 + wl.abs()) * EPS32).all()


def _top(c, i, t, m):
    """The largest score of each row of sequence i."""
    rep = c.q.shape[1] // c.k[i].shape[1]
    s = torch.einsum("mhd,shd->mhs", f64(c.q[t:t + m]), c.k[i].repeat_interleave(rep, 1)) * c.q.shape[-1] ** -0.5
    seen = torch.arange(len(c.k[i])) <= c.past[i] + torch.arange(m)[:, None]
    return s.masked_fill(~seen[:, None], -math.inf).amax(-1)


@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("m,lens,Hq,Hkv,D", [(1, [900, 333], 4, 2, 128), (1, [2500], 4, 4, 64), (3, [700, 64], 8, 2, 64), (8, [600], 6, 2, 128),
                                               (2, [24, 40, 9, 30], 16, 4, 128)])
def test_decode_weights(kv, m, lens, Hq, Hkv, D):
    """Many keys of about equal weight, whose values nearly cancel: an output is small beside what went into it."""
    c = ref.Case([m] * len(lens), [x - m for x in lens], Hq, Hkv, D, 32, BF16, kv, seed=50 + m)
    c.q.mul_(0.25)
    c.qd.copy_(c.q)
    out, lse = kda.attn_decode_multi(c.qd.view(len(lens), m, Hq, D), *c.cache, want_lse=True, **c.scales)
    _sharp(c, out, lse, kv)


# ---------------------------------------------------------------- lengths out of range, cut items of odd groups
@pytest.mark.parametrize("dtype,kv", KV)
def test_clamped_lengths(dtype, kv):
    """A length beyond the table is all of the table, pages without a number read as zeros; a negative one is no key."""
    m, Hq, Hkv, D, page = 2, 4, 2, 64, 16
    c = ref.Case([m] * 3, [100, 50, 70], Hq, Hkv, D, page, dtype, kv, seed=6)
    k, v, table, lens = c.cache
    q = c.qd.view(3, m, Hq, D)

    def both(n):
        n = i32(n)
        return (*kda.attn_decode_multi(q, k, v, table, n, want_lse=True, **c.scales),
                *kda.attn_prefill_paged(c.qd, k, v, table, n, c.cu, want_lse=True, **c.scales))

    full = c.cols * page
    # (the page that sequence 1's 52 tokens do not fill holds NaN behind them: the table ends before it)
    whole = 52 // page * page
    t = table.clone()
    t[1, whole // page:] = -1
    kk, vv = ([x[0], torch.cat([x[1][:whole], torch.zeros(full - whole, Hkv, D, dtype=F64)]), x[2]] for x in (c.k, c.v))
    for n in (full, full + 1, 2 ** 31 - 1):
        st, length = word(), i32([102, n, 72])
        out, lse = kda.attn_decode_multi(q, k, v, t, length, want_lse=True, status=st, **c.scales)
        pre, pl = kda.attn_prefill_paged(c.qd, k, v, t, length, c.cu, want_lse=True, **c.scales)
        assert int(st) == INVALID
        for o, x in ((out, lse), (pre, pl)):
            ref.check(o, x, c.q, kk, vv, c.lens, [100, full - m, 70])
    for n in (-5, -2 ** 31, 0):
        out, lse, pre, pl = both([102, n, 72])
        assert (out[1] == 0).all() and (pre[m:2 * m] == 0).all()
        assert torch.isneginf(lse[1]).all() and torch.isneginf(pl[m:2 * m]).all()


@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(3, 1, 64), (5, 5, 128)])
def test_cut_items_of_odd_groups(kv, Hq, Hkv, D):
    """Two blocks of queries an item, cut along the keys, the last block partly or not there."""
    c = ref.Case([200, 3, 300, 100], [3000, 2500, 500, 1700], Hq, Hkv, D, 64, BF16, kv, seed=51)
    out, lse = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, **c.scales)
    c.check(out, lse)


# ---------------------------------------------------------------- codes of keys
@pytest.mark.parametrize("D,page,R,inter,fused", [(64, 16, 64, False, True), (64, 256, 32, True, True), (64, 64, 10, False, False),
                                                  (128, 16, 64, True, True)])
def test_append_codes_are_the_nearest(D, page, R, inter, fused):
    """Of ragged sequences, rows that are parts of wider ones, and heads of 64: scales and codes of the exact rotation, to what
    the angle and the cosine are off by (2^-26 of the pair)."""
    from test_gpu_attn import _appended
    x = _appended(BF16, "e4m3", D, page, [900, 1, 0, 517], [33, 5000, 2, 250], R=R, inter=inter, fused=fused, seed=52)
    n = x["live"]
    pg, place = x["table"][x["ids"][:n].long(), x["pos"][:n].long() // page].long(), x["pos"][:n].long() % page
    src = f64(x["k"])[:n]
    want = ref.rotate(src, x["pos"][:n], x["freq"], inter, 1.0)
    s, got = f64(x["scales"][0])[pg, :, place], f64(x["caches"][0].float())[pg, :, place]
    assert torch.equal(s, ref.scale_of(want))
    y = want / s[..., None]
    half = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 4)
    size = _size(src, R, inter, 1.0)
    size[..., R:] = 0
    assert ((got - y).abs() <= half + 2.0 ** -26 * size / s[..., None]).all()
    assert torch.equal(got[..., R:], ref.codes(want, s)[..., R:])
