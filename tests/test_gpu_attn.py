"""The attention layers against their float64 definitions (tests/attn_reference.py): rotation and cache writes, packed and
paged prefill, decode of one and several tokens."""
import math

import pytest
import torch

import attn_reference as ref
from attn_reference import EPS16, EPS32, F8, F64, f64
from linear_attention_serving_k1_gb300 import kda

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
INVALID = kda.STATUS_CODES["KDA_ERR_INVALID_ARG"]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- rotation
def _near(got, want, size, dtype, angle=2.0 ** -22):
    """A rotated element: two products and a sum in fp32 (3 roundings), an angle right to `angle`, one rounding of the
    result; `size`: the magnitude of its pair."""
    tol = (angle + 6 * EPS32) * size + (EPS16 if dtype == BF16 else EPS32) * want.abs() + 1e-37
    assert ((f64(got) - want).abs() <= tol).all(), float(((f64(got) - want).abs() / tol).max())


def _size(x, R, interleaved, scale):
    """Magnitude of each element's pair."""
    i = torch.arange(R // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y = x.abs().clone()
    y[..., ia] = y[..., ib] = (x[..., ia].abs() + x[..., ib].abs()) * max(scale, 1.0)
    return y


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,R,inter,scale", [(128, 128, False, 1.0), (128, 64, True, 1.25), (64, 64, True, 1.0), (64, 32, False, 0.5),
                                             (128, 6, False, 1.0), (64, 10, True, 1.0), (128, 24, False, 1.0), (64, 2, False, 1.0),
                                             (128, 0, False, 1.0)])
def test_rotation(dtype, D, R, inter, scale):
    T, Hq, Hkv = 37, 5, 1
    g = torch.Generator().manual_seed(R)
    q, k = (torch.randn(T, h, D, generator=g).to(dtype) for h in (Hq, Hkv))
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[:3] = torch.tensor([0, 1, (1 << 20) - 1])
    freq = kda.rope_frequencies(R, 500000.0)[0] if R else None
    qo, ko = kda.kv_append(q.cuda(), k.cuda(), None, pos.cuda(), inv_freq=freq.cuda() if R else None, interleaved=inter,
                           rope_scale=scale)
    for got, x in ((qo, f64(q)), (ko, f64(k))):
        if not R:
            assert torch.equal(f64(got), x)
            continue
        _near(got, ref.rotate(x, pos, freq, inter, scale), _size(x, R, inter, scale), dtype)
        assert torch.equal(f64(got)[..., R:], x[..., R:])


@pytest.mark.parametrize("top,angle", [(1 << 24, 2.0 ** -22), (2 ** 31 - 1, 2.0 ** -15)])
def test_rotation_far_out(top, angle):
    """Positions up to the largest int32."""
    T, D = 200, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 2, D, generator=g)
    pos = torch.randint(top // 2, top, (T,), generator=g, dtype=torch.int32)
    pos[0] = top
    freq, _ = kda.rope_frequencies(D, 10000.0)
    got, _ = kda.kv_append(x.cuda(), x.cuda(), None, pos.cuda(), inv_freq=freq.cuda(), want_k=False)
    _near(got, ref.rotate(f64(x), pos, freq, False, 1.0), _size(f64(x), D, False, 1.0), FP32, angle)


def _appended(dtype, kv, D, page, lens, past, Hq=4, Hkv=2, R=32, inter=False, fused=False, pad=3, seed=0, values=None):
    """One append of ragged sequences; returns what it had and what it wrote."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens) + pad, len(lens)
    rows = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g)
    if values is not None:
        rows[:, Hq * D:] = values(rows[:, Hq * D:])
    rows = rows.to(dtype)
    q, k, v = (x.view(T, -1, D) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 1))
    ids = torch.cat([torch.full((L,), n, dtype=torch.int32) for n, L in enumerate(lens)] + [torch.full((pad,), -1, dtype=torch.int32)])
    pos = torch.cat([torch.arange(p, p + L, dtype=torch.int32) for p, L in zip(past, lens)] + [torch.full((pad,), -1, dtype=torch.int32)])
    need = [-(-(L + p) // page) for L, p in zip(lens, past)]
    pages = sum(need) + 2
    order, at = torch.randperm(pages, generator=g).to(torch.int32), 0
    table = torch.full((N, max(need) + 1), -1, dtype=torch.int32)
    for n in range(N):
        table[n, :need[n]] = order[at:at + need[n]]
        at += need[n]
    shape = (pages, Hkv, page, D)
    if kv == "e4m3":
        caches = [torch.full(shape, 3.0).to(F8).cuda() for _ in range(2)]
        scales = [torch.full(shape[:3], 5.0).cuda() for _ in range(2)]
    else:
        caches, scales = [torch.full(shape, 7.0, dtype=dtype).cuda() for _ in range(2)], [None, None]
    d = rows.cuda()
    qd, kd, vd = (x.view(T, -1, D) for x in d.split([Hq * D, Hkv * D, Hkv * D], 1))
    if not fused:
        qd, kd, vd = qd.contiguous(), kd.contiguous(), vd.contiguous()
    freq, _ = kda.rope_frequencies(R, 10000.0)
    qo, ko, st = torch.full((T, Hq, D), 9.0, dtype=dtype).cuda(), torch.full((T, Hkv, D), 9.0, dtype=dtype).cuda(), word()
    kda.kv_append(qd, kd, vd, pos.cuda(), seq_ids=ids.cuda(), page_table=table.cuda(), k_cache=caches[0], v_cache=caches[1],
                  k_scale=scales[0], v_scale=scales[1], inv_freq=freq.cuda(), interleaved=inter, q_out=qo, k_out=ko, status=st)
    return dict(q=q, k=k, v=v, pos=pos, ids=ids, table=table, caches=caches, scales=scales, qo=qo, ko=ko, status=int(st), freq=freq,
                live=sum(lens))


@pytest.mark.parametrize("dtype,kv", [(BF16, "same"), (BF16, "e4m3"), (FP32, "same")])
@pytest.mark.parametrize("D,page,inter,fused", [(128, 64, False, False), (64, 16, True, True), (128, 16, True, True), (64, 256, False, True)])
def test_append(dtype, kv, D, page, inter, fused):
    """Rows of queries, keys and the cache; every other place of them as it was."""
    x = _appended(dtype, kv, D, page, [1, 0, 70, 17], [33, 5, 0, 250], inter=inter, fused=fused)
    n, R = x["live"], 32
    assert x["status"] == 0
    for name, out in (("q", "qo"), ("k", "ko")):
        src = f64(x[name])[:n]
        want = ref.rotate(src, x["pos"][:n], x["freq"], inter, 1.0)
        _near(x[out][:n], want, _size(src, R, inter, 1.0), dtype)
        assert (f64(x[out])[n:] == 9).all()
    pg, place = x["table"][x["ids"][:n].long(), x["pos"][:n].long() // page].long(), x["pos"][:n].long() % page
    for i, name in enumerate("kv"):
        c = f64(x["caches"][i].float())
        got = c[pg, :, place].clone()
        other = torch.ones(c.shape[:3], dtype=torch.bool)
        other[pg, :, place] = False
        assert (c[other] == (3 if kv == "e4m3" else 7)).all()
        src = f64(x[name])[:n]
        want = ref.rotate(src, x["pos"][:n], x["freq"], inter, 1.0) if name == "k" else src
        if kv != "e4m3":
            if name == "k":
                assert torch.equal(got, f64(x["ko"])[:n])
            else:
                assert torch.equal(got, src)
            continue
        s = f64(x["scales"][i])[pg, :, place]
        assert (f64(x["scales"][i])[other] == 5).all()
        if name == "v":
            assert torch.equal(s, ref.scale_of(src)) and torch.equal(got, ref.codes(src, s))
        else:   # keys are rotated in fp32 first: half a step of e4m3 (2^-4; 2^-10 s below 2^-6 s), and the rotation's error
            assert ((s / ref.scale_of(want)).log2().abs() <= 1).all() and (s.log2() == s.log2().round()).all()
            size = _size(src, R, inter, 1.0)
            assert ((got * s[..., None] - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * s[..., None] + 2.0 ** -19 * size).all()


@pytest.mark.parametrize("R,inter,scale", [(128, False, 1.2079441), (128, True, 1.0), (24, False, 1.0)])
def test_append_rows_of_eight_bits_are_the_nearest(R, inter, scale):
    """Of 4 million keys, codes and scales are those of the exact rotation, to what the angle and the cosine are off by
    (2^-26 of the pair); elements that are not rotated and the first position (cosine 1) lie on halves often."""
    T, H, D, page = 4000, 8, 128, 64
    g = torch.Generator().manual_seed(R + inter)
    k = torch.randn(T, H, D, generator=g).to(BF16)
    pos = torch.arange(T, dtype=torch.int32)
    freq, _ = kda.rope_frequencies(R, 500000.0)
    n = -(-T // page)
    cache = [torch.zeros(n, H, page, D, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
    sc = [torch.zeros(n, H, page, device="cuda") for _ in range(2)]
    kd = k.cuda()
    kda.kv_append(None, kd, kd, pos.cuda(), seq_ids=torch.zeros_like(pos).cuda(), page_table=torch.arange(n, dtype=torch.int32)[None].cuda(),
                  k_cache=cache[0], v_cache=cache[1], k_scale=sc[0], v_scale=sc[1], inv_freq=freq.cuda(), interleaved=inter, rope_scale=scale)
    flat = lambda x: f64(x.float()).transpose(1, 2).reshape(n * page, H, -1)[:T]  # noqa: E731
    scale32 = float(torch.tensor(scale, dtype=FP32))
    want = ref.rotate(f64(k), pos, freq, inter, scale32)
    got, s = flat(cache[0]), flat(sc[0][..., None])[..., 0]
    assert torch.equal(s, ref.scale_of(want))
    y = want / s[..., None]
    half = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 4)
    size = _size(f64(k), R, inter, scale32)
    size[..., R:] = 0
    assert ((got - y).abs() <= half + 2.0 ** -26 * size / s[..., None]).all()
    exact = torch.ones(T, H, D, dtype=torch.bool)
    exact[int(scale == 1.0):, :, :R] = False
    assert torch.equal(got[exact], ref.codes(want, s)[exact])


def test_append_in_place_and_into_the_cache_alone():
    x = _appended(BF16, "same", 128, 64, [20], [100], pad=0)
    q, k, v = (x[n].cuda().contiguous() for n in "qkv")
    kda.kv_append(q, k, None, x["pos"].cuda(), inv_freq=x["freq"].cuda(), q_out=q, k_out=k)
    assert torch.equal(q, x["qo"]) and torch.equal(k, x["ko"])
    cache = [torch.full_like(c, 7.0) for c in x["caches"]]
    qo, ko = kda.kv_append(None, x["k"].cuda().contiguous(), v, x["pos"].cuda(), seq_ids=x["ids"].cuda(), page_table=x["table"].cuda(),
                           k_cache=cache[0], v_cache=cache[1], inv_freq=x["freq"].cuda())
    assert qo is None and ko is None and all(torch.equal(a, b) for a, b in zip(cache, x["caches"]))
    kda.kv_append(q[:0], k[:0], v[:0], x["pos"][:0].cuda())


def test_append_rows_of_eight_bits_at_the_ends_of_their_range():
    """Zero rows, the smallest and largest values, 448 and just above, values that are not finite."""
    special = [0.0, 2.0 ** -133, 448.0, 450.0, 3.0e38, 2.0 ** -118]

    def values(t):
        t = t.clone()
        for i, s in enumerate(special):
            t[i] = s * torch.sign(t[i])
        t[6, 5], t[7, 70], t[8, 3], t[8, 4] = math.inf, math.nan, -math.inf, math.nan
        return t

    x = _appended(BF16, "e4m3", 64, 16, [12], [0], R=2, values=values, pad=0, Hkv=1)
    v, s, c = f64(x["v"]), f64(x["scales"][1]), f64(x["caches"][1].float())
    pg = x["table"][0, 0].long()
    want = ref.scale_of(v)[:, 0]
    got = s[pg, 0, :12]
    assert torch.equal(got.isnan(), want.isnan()) and int(want.isnan().sum()) == 1 and want[7].isnan()   # (v's row of element 70)
    fine = ~want.isnan()
    assert torch.equal(got[fine], want[fine])
    assert torch.equal(c[pg, 0, :12][fine], ref.codes(v[fine, 0], want[fine]))
    # (key 4 too: turned by 4 radians its pair reaches 3e38 (|cos 4| + |sin 4|) = 4.2e38, beyond fp32)
    assert f64(x["scales"][0])[pg, 0, :12].isnan().nonzero().flatten().tolist() == [4, 6, 8]


def test_append_rows_without_a_page():
    """Behind the table, and page numbers out of range: reported, rotated, not stored."""
    x = _appended(BF16, "same", 64, 16, [40], [0], pad=0)
    q, k, v = (x[n].cuda().contiguous() for n in "qkv")
    table = x["table"].clone()
    for change in ((0, 1, 1 << 20), (0, 1, -7), (0, 1, int(x["caches"][0].shape[0]))):
        t = table.clone()
        t[change[0], change[1]] = change[2]
        cache, st = [torch.full_like(c, 7.0) for c in x["caches"]], word()
        qo, _ = kda.kv_append(q, k, v, x["pos"].cuda(), seq_ids=x["ids"].cuda(), page_table=t.cuda(), k_cache=cache[0], v_cache=cache[1],
                              inv_freq=x["freq"].cuda(), status=st)
        assert int(st) == INVALID and torch.equal(qo, x["qo"])
        want = x["caches"][0].clone()
        want[table[0, 1].long()] = 7.0
        assert torch.equal(cache[0], want)
    st, cache = word(), [torch.full_like(c, 7.0) for c in x["caches"]]
    kda.kv_append(q, k, v, x["pos"].cuda() + (1 << 30), seq_ids=x["ids"].cuda(), page_table=table.cuda(), k_cache=cache[0], v_cache=cache[1], status=st)
    assert int(st) == INVALID and (cache[0] == 7).all()
    ids = x["ids"].cuda() + 1                      # no such sequence: padding
    qo = torch.full_like(q, 9.0)
    kda.kv_append(q, k, v, x["pos"].cuda(), seq_ids=ids, page_table=table.cuda(), k_cache=cache[0], v_cache=cache[1], q_out=qo)
    assert (cache[0] == 7).all() and (qo == 9).all()


# ---------------------------------------------------------------- packed prompts
def _packed(lens, Hq, Hkv, D, dtype, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    q = (2 * torch.randn(T + pad, Hq, D, generator=g)).to(dtype)
    k = (torch.randn(T + pad, Hkv, D, generator=g) * (1 + 3 * (torch.arange(D) % 29 == 3))).to(dtype)
    v = torch.randn(T + pad, Hkv, D, generator=g).to(dtype)
    return q, k, v, torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _check_packed(out, lse, q, k, v, lens, scale=None):
    T = sum(lens)
    split = lambda x: list(f64(x)[:T].split(list(lens)))  # noqa: E731
    ref.check(out[:T], lse[:T], q[:T], split(k), split(v), lens, [0] * len(lens), scale)


PACKED = [
    ([1], 1, 1, 64), ([2], 8, 2, 128), ([300], 4, 2, 128), ([128], 2, 1, 64), ([129, 127], 2, 2, 128), ([256, 1, 0, 130], 4, 1, 64),
    ([0, 0, 65, 3, 0], 3, 1, 128), ([64, 511], 6, 2, 128), ([513], 5, 5, 64), ([1] * 40 + [200], 2, 2, 128), ([385], 8, 1, 64),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens,Hq,Hkv,D", PACKED)
def test_prefill(dtype, lens, Hq, Hkv, D):
    q, k, v, cu = _packed(lens, Hq, Hkv, D, dtype)
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, q, k, v, lens)


@pytest.mark.parametrize("lens", [[65] * 40, [1300, 1, 700, 300, 500]])
def test_prefill_of_many_items(lens):
    """More blocks and heads than four an SM: no item is cut along its keys."""
    q, k, v, cu = _packed(lens, 64, 32, 64, BF16, 8)
    assert (sum(lens) + 127) // 128 * 32 >= 4 * 152
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, q, k, v, lens)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens", [[i % 3 for i in range(2200)], [(7 * i) % 11 for i in range(150)] + [300]])
def test_prefill_of_many_sequences(dtype, lens):
    """More than the plan keeps in shared memory, and more than its warps."""
    q, k, v, cu = _packed(lens, 2, 1, 64, dtype, 15)
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, q, k, v, lens)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefill_options(dtype):
    """Equal sequences without offsets, a scale, outputs of the caller's, a hint; equal calls give equal bits."""
    q, k, v, cu = _packed([150, 150], 4, 2, 128, dtype, 1)
    d = [x.cuda() for x in (q, k, v)]
    out, lse = kda.attn_prefill(*d, num_seqs=2, scale=0.03, want_lse=True)
    _check_packed(out, lse, q, k, v, [150, 150], 0.03)
    o2, l2 = torch.full_like(out, 5.0), torch.full_like(lse, 5.0)
    a, b = kda.attn_prefill(*d, cu, scale=0.03, out=o2, lse=l2, max_seq_len=150)
    assert a is o2 and b is l2 and torch.equal(o2, out) and torch.equal(l2, lse)
    o3, none = kda.attn_prefill(*d, cu, scale=0.03)
    assert none is None and torch.equal(o3, out)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefill_leaves_rows_behind_the_last_sequence(dtype):
    """A padded batch whose padding is NaN, and malformed offsets."""
    lens = [100, 31]
    q, k, v, cu = _packed(lens, 4, 2, 64, dtype, 2, pad=9)
    q[131:], k[131:], v[131:] = math.nan, math.nan, math.nan
    d = [x.cuda() for x in (q, k, v)]
    out, lse = torch.full_like(d[0], 5.0), torch.full(q.shape[:2], 5.0).cuda()
    ws = torch.empty(kda.attn_workspace_size(kda.make_attn_desc(140, 4, 2, 64, 2, 0 if dtype == BF16 else 1)), dtype=torch.uint8, device="cuda")
    kda.attn_prefill(*d, cu, out=out, lse=lse, workspace=ws)
    assert kda.prefill_status(ws) == 0
    _check_packed(out, lse, q, k, v, lens)
    assert (out[131:] == 5).all() and (lse[131:] == 5).all()
    for bad in ([0, 100, 90], [1, 50, 100], [0, 100, 141], [0, -5, 100], [0, 2 ** 31 - 1, 100]):
        out.fill_(5.0)
        kda.attn_prefill(*d, i32(bad), out=out, lse=lse, workspace=ws)
        assert kda.prefill_status(ws) == INVALID and (out == 5).all(), bad


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 2), (64, 3, 3)])
def test_prefill_values_that_are_not_finite(dtype, D, Hq, Hkv):
    """They change rows of their own and later tokens of their sequence only."""
    lens = [200, 150]
    q, k, v, cu = _packed(lens, Hq, Hkv, D, dtype, 3)
    base, _ = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu)
    for bad in (math.nan, math.inf, -math.inf):
        x = v.clone()
        x[70, 0, 5], x[130, Hkv - 1, 9], x[199, 0, 0] = bad, bad, bad
        out, lse = kda.attn_prefill(q.cuda(), k.cuda(), x.cuda(), cu, want_lse=True)
        wrong = ~torch.isfinite(out)
        want = torch.zeros_like(wrong)
        rep = Hq // Hkv
        want[70:200, :rep, 5] = True
        want[130:200, -rep:, 9] = True
        want[199, :rep, 0] = True
        assert torch.equal(wrong, want), bad
        assert torch.equal(out[~want], base[~want]) and torch.isfinite(lse).all()
    x = k.clone()
    x[70, 0, 5] = math.nan
    out, _ = kda.attn_prefill(q.cuda(), x.cuda(), v.cuda(), cu)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[70:200, :Hq // Hkv] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], base[~want])
    x = q.clone()
    x[70, 1] = math.nan
    out, _ = kda.attn_prefill(x.cuda(), k.cuda(), v.cuda(), cu)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[70, 1] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], base[~want])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefill_large_and_small_scores(dtype):
    """Rows whose maximum grows by hundreds from tile to tile, and rows of equal keys."""
    lens, D = [500], 64
    q, k, v, cu = _packed(lens, 2, 1, D, dtype, 4)
    k = (k.float() * torch.linspace(0.01, 12, 500)[:, None, None]).to(dtype)
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, q, k, v, lens)
    k = k.flip(0).contiguous()
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, q, k, v, lens)
    out, lse = kda.attn_prefill(torch.zeros_like(q).cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, torch.zeros_like(q), k, v, lens)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefill_of_many_heads(dtype, D):
    """Blocks and heads enough for the whole GPU (fp32: CTAs of 64 rows), packed and over a cache, values not finite."""
    lens, Hq, Hkv = [200, 1, 0, 150], 160, 80
    q, k, v, cu = _packed(lens, Hq, Hkv, D, dtype, 17)
    out, lse = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, want_lse=True)
    _check_packed(out, lse, q, k, v, lens)
    x = v.clone()
    x[70, 3, 5], x[199, 79, 0] = math.nan, math.inf
    got, _ = kda.attn_prefill(q.cuda(), k.cuda(), x.cuda(), cu)
    want = torch.zeros_like(got, dtype=torch.bool)
    want[70:200, 6:8, 5], want[199, 158:, 0] = True, True
    assert torch.equal(~torch.isfinite(got), want) and torch.equal(got[~want], out[~want])
    c = ref.Case(lens, [60, 0, 7, 300], Hq, Hkv, D, 32, dtype, "same", seed=18)
    out, lse = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True)
    c.check(out, lse)


# ---------------------------------------------------------------- over the cache
KV = [(BF16, "same"), (BF16, "e4m3"), (FP32, "same")]
BEHIND = [
    ([5, 130], [0, 200], 4, 2, 128, 64), ([1, 0, 64], [127, 50, 1], 4, 1, 64, 16), ([100], [29], 6, 2, 128, 32),
    ([260, 3], [77, 500], 3, 3, 64, 128), ([7, 9], [-3, 0], 2, 1, 128, 16), ([4], [-4], 2, 2, 64, 16), ([33], [1000], 8, 2, 128, 1024),
]


@pytest.mark.parametrize("dtype,kv", KV)
@pytest.mark.parametrize("lens,past,Hq,Hkv,D,page", BEHIND)
def test_prefill_paged(dtype, kv, lens, past, Hq, Hkv, D, page):
    """Places of the cache that no sequence holds are NaN."""
    c = ref.Case(lens, past, Hq, Hkv, D, page, dtype, kv)
    out, lse = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, **c.scales)
    c.check(out, lse)


@pytest.mark.parametrize("dtype,kv", KV)
@pytest.mark.parametrize("m,lens,Hq,Hkv,D,page", [
    (1, [1], 1, 1, 64, 16), (1, [0, 1, 15, 16, 17, 64, 300], 4, 2, 128, 16), (1, [2000, 3], 8, 1, 128, 64), (1, [700] * 9, 6, 2, 64, 32),
    (2, [1, 2, 40, 0], 4, 4, 64, 16), (4, [4, 3, 129, 500], 8, 2, 128, 32), (5, [70, 6], 24, 2, 64, 64), (8, [1000], 16, 2, 128, 128),
    (3, [513, 33], 20, 1, 128, 16), (1, [90], 40, 1, 64, 256),
])
def test_decode(dtype, kv, m, lens, Hq, Hkv, D, page):
    c = ref.Case([m] * len(lens), [x - m for x in lens], Hq, Hkv, D, page, dtype, kv, seed=m)
    st = word()
    q = c.qd.view(len(lens), m, Hq, D)
    if m == 1:
        out, lse = kda.attn_decode(q[:, 0], *c.cache, want_lse=True, status=st, **c.scales)
    else:
        out, lse = kda.attn_decode_multi(q, *c.cache, want_lse=True, status=st, **c.scales)
    # (a length below m: its table cannot say so, the case's lengths are clamped at 0)
    c.check(out, lse)
    assert int(st) == 0


@pytest.mark.parametrize("dtype,kv", KV)
@pytest.mark.parametrize("m", [1, 2])
def test_decode_of_many_sequences(dtype, kv, m):
    """More sequences than threads that look for a share's start, among them empty ones."""
    lens = [(13 * i) % 40 for i in range(300)]
    c = ref.Case([m] * 300, [x - m for x in lens], 2, 1, 64, 16, dtype, kv, seed=16)
    out, lse = kda.attn_decode_multi(c.qd.view(300, m, 2, 64), *c.cache, want_lse=True, **c.scales)
    c.check(out, lse)
    pre, pl = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, **c.scales)
    c.check(pre, pl)


@pytest.mark.parametrize("dtype,kv", KV)
def test_empty_batches_and_a_cache_without_a_page(dtype, kv):
    """No sequence, no new token, and lengths whose pages do not exist: zeros, as keys and values are, and reported."""
    c = ref.Case([3, 3], [50, 5], 4, 2, 64, 16, dtype, kv, seed=14)
    k, v, table, lens = c.cache
    none = {n: s[:0] if s is not None else None for n, s in c.scales.items()}
    out, lse = kda.attn_decode(c.qd[:0], k, v, table[:0].contiguous(), lens[:0], want_lse=True, **c.scales)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, _ = kda.attn_prefill_paged(c.qd[:0], k, v, table, lens, i32([0, 0, 0]), **c.scales)
    assert out.shape == (0, 4, 64)
    st = word()
    out, lse = kda.attn_decode_multi(c.qd.view(2, 3, 4, 64), k[:0], v[:0], table, lens, want_lse=True, status=st, **none)
    assert int(st) == INVALID and (out == 0).all()
    want = torch.tensor([[51, 52, 53], [6, 7, 8]], dtype=F64).log()[:, :, None].expand(2, 3, 4)    # scores of 0
    assert (f64(lse) - want).abs().max() < 1e-5
    out, lse = kda.attn_prefill_paged(c.qd, k[:0], v[:0], table, lens, c.cu, want_lse=True, **none)
    assert (out == 0).all() and (f64(lse).view(2, 3, 4) - want).abs().max() < 1e-5


@pytest.mark.parametrize("dtype,kv", KV)
def test_decode_values_that_are_not_finite(dtype, kv):
    """m tokens: a value of a later token does not reach an earlier one."""
    m, D, Hq, Hkv = 4, 128, 4, 2
    c = ref.Case([m, m], [200, 60], Hq, Hkv, D, 16, dtype, kv, seed=5)
    q = c.qd.view(2, m, Hq, D)
    base, bl = kda.attn_decode_multi(q, *c.cache, want_lse=True, **c.scales)
    k, v, table, lens = c.cache
    j = 202                                         # the third of sequence 0's new tokens
    pg = int(table[0, j // 16])
    want = torch.zeros_like(base, dtype=torch.bool)
    if kv == "e4m3":
        vs = c.scales["v_scale"].clone()
        vs[pg, 1, j % 16] = math.nan
        want[0, 2:, 2:] = True
        out, lse = kda.attn_decode_multi(q, k, v, table, lens, k_scale=c.scales["k_scale"], v_scale=vs, want_lse=True)
    else:
        v = v.clone()
        v[pg, 1, j % 16, 7] = math.inf
        want[0, 2:, 2:, 7] = True
        out, lse = kda.attn_decode_multi(q, k, v, table, lens, want_lse=True)
    assert torch.equal(~torch.isfinite(out), want) and torch.equal(out[~want], base[~want]) and torch.equal(lse, bl)


@pytest.mark.parametrize("dtype,kv", KV)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 3, 64)])
def test_prefill_paged_values_that_are_not_finite(dtype, kv, Hq, Hkv, D):
    """Of a new token (they reach it and the later ones), and of a cached one (they reach all)."""
    c = ref.Case([150, 20], [60, 300], Hq, Hkv, D, 32, dtype, kv, seed=11)
    base, bl = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, **c.scales)
    k, v, table, lens = c.cache
    rep = Hq // Hkv
    for j, first in ((60 + 100, 100), (7, 0)):
        pg = int(table[0, j // 32])
        want = torch.zeros_like(base, dtype=torch.bool)
        if kv == "e4m3":
            vs = c.scales["v_scale"].clone()
            vs[pg, 1, j % 32] = math.nan
            want[first:150, rep:2 * rep] = True
            out, lse = kda.attn_prefill_paged(c.qd, k, v, table, lens, c.cu, k_scale=c.scales["k_scale"], v_scale=vs, want_lse=True)
        else:
            x = v.clone()
            x[pg, 1, j % 32, 9] = math.nan
            want[first:150, rep:2 * rep, 9] = True
            out, lse = kda.attn_prefill_paged(c.qd, k, x, table, lens, c.cu, want_lse=True)
        assert torch.equal(~torch.isfinite(out), want) and torch.equal(out[~want], base[~want]) and torch.equal(lse, bl)


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_prefill_paged_cut_along_the_keys(kv):
    """Few queries behind a long past: parts, joined."""
    c = ref.Case([40, 3, 1], [6000, 0, 2500], 4, 1, 64, 64, BF16, kv, seed=12)
    out, lse = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, **c.scales)
    c.check(out, lse)


@pytest.mark.parametrize("kv", ["same", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv", [(32, 16), (33, 11)])
def test_waits_that_give_up(kv, Hq, Hkv):
    """A wait limit of one poll in a call of many long items: it returns, its status says so, and the workspace and GPU are
    as good as before."""
    c = ref.Case([2000, 5], [4000, 130], Hq, Hkv, 128, 64, BF16, kv, seed=13)
    desc = kda.make_attn_desc(2005, Hq, Hkv, 128, 2, 0, kv_dtype=2 if kv == "e4m3" else None, page_size=64, pages_per_seq=c.cols,
                              num_pages=c.cache[0].shape[0])
    ws = torch.empty(kda.attn_workspace_size(desc), dtype=torch.uint8, device="cuda")
    run = lambda **kw: kda.attn_prefill_paged(c.qd, *c.cache, c.cu, workspace=ws, want_lse=True, **c.scales, **kw)  # noqa: E731
    base, bl = run()
    assert kda.prefill_status(ws) == 0
    run(wait_limit=1)
    assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_TIMEOUT"]
    out, lse = run()
    assert kda.prefill_status(ws) == 0 and torch.equal(out, base) and torch.equal(lse, bl)


@pytest.mark.parametrize("dtype,kv", KV)
def test_lengths_and_pages_out_of_range(dtype, kv):
    """Reported; other sequences are as ever, and the sequence itself is as with a page of zeros or the clamped length."""
    m, Hq, Hkv, D = 2, 4, 2, 64
    c = ref.Case([m] * 3, [100, 50, 70], Hq, Hkv, D, 16, dtype, kv, seed=6)
    q = c.qd.view(3, m, Hq, D)
    k, v, table, lens = c.cache
    base, _ = kda.attn_decode_multi(q, *c.cache, **c.scales)
    pbase, _ = kda.attn_prefill_paged(c.qd, *c.cache, c.cu, **c.scales)
    desc = kda.make_attn_desc(3 * m, Hq, Hkv, D, 3, 0 if dtype == BF16 else 1, kv_dtype=2 if kv == "e4m3" else None, page_size=16,
                              pages_per_seq=c.cols, num_pages=k.shape[0])
    ws = torch.empty(max(kda.attn_workspace_size(desc), kda.attn_workspace_size(desc, decode=True)), dtype=torch.uint8, device="cuda")

    def both(t, n):
        st = word()
        out, _ = kda.attn_decode_multi(q, k, v, t, n, status=st, **c.scales)
        pre, _ = kda.attn_prefill_paged(c.qd, k, v, t, n, c.cu, workspace=ws, **c.scales)
        assert int(st) == INVALID and kda.prefill_status(ws) == INVALID
        for o, b in ((out, base), (pre.view_as(out), pbase.view_as(out))):
            assert torch.equal(o[0], b[0]) and torch.equal(o[2], b[2])
        return out, pre

    for number in (-1, int(k.shape[0]), 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 1] = number
        out, pre = both(t, lens)
        kk, vv = [x.clone() for x in c.k], [x.clone() for x in c.v]
        kk[1][16:32], vv[1][16:32] = 0, 0
        for o in (out, pre):
            ref.check(o, None, c.q, kk, vv, c.lens, c.past)
    out, _ = both(table, i32([102, -5, 72]))
    assert (out[1] == 0).all()
    both(table, i32([102, 2 ** 31 - 1, 72]))


def test_together():
    """A serving step over one cache: plan, append, prompt attention (packed, and behind a cached past), then decode steps;
    the same tokens at once and bit by bit."""
    Hq, Hkv, D, page, lens = 8, 2, 128, 16, [70, 1, 33]
    g = torch.Generator().manual_seed(9)
    more = 4                                         # tokens decoded one by one
    x = [torch.randn(n + more, Hq + 2 * Hkv, D, generator=g).to(BF16) for n in lens]
    freq, scale = kda.rope_frequencies(D, 10000.0, scaling="parts", factor=4.0, original_len=64)
    full = [ref.rotate(f64(t[:, :Hq + Hkv]), torch.arange(len(t)), freq, False, scale).to(BF16) for t in x]
    q, k, v = [f[:, :Hq] for f in full], [f64(f[:, Hq:]) for f in full], [f64(t[:, Hq + Hkv:]) for t in x]
    pages = [-(-len(t) // page) for t in x]
    table = torch.full((3, max(pages)), -1, dtype=torch.int32)
    order = torch.randperm(sum(pages), generator=g).to(torch.int32)
    for n, a in enumerate(torch.tensor([0] + pages).cumsum(0)[:-1].tolist()):
        table[n, :pages[n]] = order[a:a + pages[n]]
    table = table.cuda()
    kc, vc = (torch.full((sum(pages), Hkv, page, D), math.nan, dtype=BF16, device="cuda") for _ in range(2))

    def step(tokens, past):
        """Append `tokens` rows of every sequence; returns the plan, rotated queries and packed keys and values."""
        rows = torch.cat([t[p:p + n] for t, p, n in zip(x, past, tokens)]).cuda()
        plan = kda.plan_batch(i32(tokens), i32([0, 1, 2]), total_tokens=len(rows) + 2, past=i32(past))
        rows = torch.cat([rows, torch.full_like(rows[:2], math.nan)])
        a, b, c = (rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:])
        qo, ko = kda.kv_append(a, b, c, plan.positions, seq_ids=plan.seq_ids, page_table=table, k_cache=kc, v_cache=vc,
                               inv_freq=freq.cuda(), rope_scale=scale, want_k=True)
        return plan, qo, ko, c.contiguous()

    plan, qo, ko, vo = step(lens, [0, 0, 0])
    T = sum(lens)
    out, lse = kda.attn_prefill(qo, ko, vo, plan.cu_seqlens, want_lse=True)
    over, lse2 = kda.attn_prefill_paged(qo, kc, vc, table, i32(lens), plan.cu_seqlens, want_lse=True)
    cut = lambda y: [a[:n] for a, n in zip(y, lens)]  # noqa: E731
    ends = [torch.cat(cut(q)), cut(k), cut(v), lens, [0, 0, 0]]
    # (rows of the call round rotated values as the reference does but for ties: compare on the call's own)
    mine = list(f64(ko)[:T].split(lens))
    assert all((a - b).abs().max() <= 2.0 ** -7 * b.abs().max() for a, b in zip(mine, ends[1]))
    ref.check(out[:T], lse[:T], qo[:T].cpu(), mine, ends[2], lens, ends[4])
    ref.check(over[:T], lse2[:T], qo[:T].cpu(), mine, ends[2], lens, ends[4])
    for i in range(more):
        past = [n + i for n in lens]
        plan, qo, ko, _ = step([1, 1, 1], past)
        out, lse = kda.attn_decode(qo[:3], kc, vc, table, i32([p + 1 for p in past]), want_lse=True)
        mine = [torch.cat([a, f64(ko)[n:n + 1]]) for n, a in enumerate(mine)]
        ref.check(out, lse, qo[:3].cpu(), mine, [t[:p + 1] for t, p in zip(v, past)], [1, 1, 1], past)
    # the last tokens again, as a verify step of four drafted tokens would
    q4 = torch.stack([f[n:n + more] for f, n in zip(q, lens)]).cuda()
    out, lse = kda.attn_decode_multi(q4, kc, vc, table, i32([n + more for n in lens]), want_lse=True)
    ref.check(out, lse, q4.cpu().flatten(0, 1), mine, v, [more] * 3, lens)


# ---------------------------------------------------------------- streams, graphs, sizes
def _calls(dtype, kv, seed):
    c = ref.Case([3, 3], [700, 90], 8, 2, 128, 32, dtype, kv, seed=seed)
    q = c.qd.view(2, 3, 8, 128)
    x = _packed([150, 40], 8, 2, 128, dtype, seed)
    d = [t.cuda() for t in x[:3]]
    return [lambda **kw: kda.attn_decode_multi(q, *c.cache, want_lse=True, **c.scales, **kw),
            lambda **kw: kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, **c.scales, **kw),
            lambda **kw: kda.attn_prefill(*d, x[3], want_lse=True, **kw)]


@pytest.mark.parametrize("dtype,kv", KV)
def test_two_calls_at_once(dtype, kv):
    """On two streams, each with its own workspace, many times: the same bits as one after the other."""
    calls = [_calls(dtype, kv, s) for s in (1, 2)]
    want = [[f() for f in c] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append([f() for f in calls[i]])
    for i, s in enumerate(streams):
        got[i].append([f(stream=s) for f in calls[i]])
    torch.cuda.synchronize()
    for i in range(2):
        for results in got[i]:
            for (o, l), (a, b) in zip(results, want[i]):
                assert torch.equal(o, a) and torch.equal(l, b)


@pytest.mark.parametrize("dtype,kv", KV)
def test_captured_calls_that_share_a_workspace(dtype, kv):
    """Two graphs over one workspace, replayed in turn, with other lengths and queries in the buffers than at capture."""
    cases = [ref.Case([2, 2], p, 8, 2, 64, 16, dtype, kv, seed=s) for s, p in ((1, [600, 30]), (2, [100, 333]))]
    desc = [kda.make_attn_desc(4, 8, 2, 64, 2, 0 if dtype == BF16 else 1, kv_dtype=2 if kv == "e4m3" else None, page_size=16,
                               pages_per_seq=c.cols, num_pages=c.cache[0].shape[0]) for c in cases]
    ws = torch.empty(max(kda.attn_workspace_size(d, x) for d in desc for x in (False, True)), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c in cases:
        q = c.qd.view(2, 2, 8, 64)
        run = lambda: (kda.attn_decode_multi(q, *c.cache, want_lse=True, workspace=ws, **c.scales),  # noqa: E731
                       kda.attn_prefill_paged(c.qd, *c.cache, c.cu, want_lse=True, workspace=ws, **c.scales))
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    lens = [c.cache[3].clone() for c in cases]
    for c in cases:
        c.cache[3].copy_(i32([2, 5]))
    for g in graphs:
        g.replay()
    for c, n in zip(cases, lens):
        c.cache[3].copy_(n)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, pair in zip(cases, outs):
        for o, l in pair:
            c.check(o.reshape(c.q.shape), l.reshape(c.q.shape[:2]))


def test_workspace_stream_and_device_are_checked():
    calls = _calls(BF16, "same", 3)
    for f in calls:
        with pytest.raises(ValueError, match="workspace"):
            f(workspace=torch.empty(1 << 20, dtype=torch.uint8))
        with pytest.raises(kda.KDAError) as e:
            f(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        assert e.value.code == kda.STATUS_CODES["KDA_ERR_WORKSPACE"]
    q = torch.zeros(4, 2, 128, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="k must be"):
        kda.attn_prefill(q, q[:3], q)
    with pytest.raises(ValueError, match="must be"):
        kda.attn_prefill(q, q.float(), q)
    with pytest.raises(ValueError, match="contiguous"):
        kda.attn_prefill(q, q.transpose(0, 1).contiguous().transpose(0, 1), q)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kv_append(q, q.transpose(0, 1).contiguous().transpose(0, 1), q, i32([0, 1, 2, 3]))
    with pytest.raises(ValueError, match="overlap"):
        kda.kv_append(q, q[:1].expand(4, 2, 128), q, i32([0, 1, 2, 3]))
    with pytest.raises(ValueError, match="needs page_table"):
        kda.kv_append(q, q, q, i32([0, 1, 2, 3]), k_cache=torch.zeros(1, 2, 16, 128, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="cache must be"):
        kda.attn_decode(q, *(torch.zeros(1, 2, 16, 128, device="cuda") for _ in range(2)), i32([[0]] * 4), i32([1] * 4))


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_cache_beyond_32_bits(kv):
    """A cache of more than 2^31 elements: the last pages as in a small one."""
    Hkv, D, page = 16, 128, 64
    pages = 2 ** 31 // (Hkv * D * page) + 40
    c = ref.Case([2, 2], [130, 70], 32, Hkv, D, page, BF16, kv, seed=4)
    k, v, table, lens = c.cache
    n = k.shape[0]
    big = []
    for x in (k, v, *(s for s in c.scales.values() if s is not None)):
        y = torch.zeros(pages, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[-n:] = x
        big.append(y)
    t = torch.where(table >= 0, table + pages - n, table)
    s = dict(k_scale=big[2], v_scale=big[3]) if kv == "e4m3" else {}
    q = c.qd.view(2, 2, 32, D)
    for f in (lambda *a, **kw: kda.attn_decode_multi(q, *a, **kw), lambda *a, **kw: kda.attn_prefill_paged(c.qd, *a, c.cu, **kw)):
        small, big_ = f(*c.cache, **c.scales)[0], f(big[0], big[1], t, lens, **s)[0]
        assert torch.equal(small, big_)
    pos, rows = i32([131, 71]), torch.randn(2, Hkv, D, device="cuda").to(BF16)
    for cache, tab, sc in (((k, v), table, c.scales), (big[:2], t, s)):
        kda.kv_append(None, rows, rows, pos, seq_ids=i32([0, 1]), page_table=tab, k_cache=cache[0], v_cache=cache[1], **sc)
    assert torch.equal(big[0][-n:].view(torch.uint8), k.view(torch.uint8)) and torch.equal(big[1][-n:].view(torch.uint8), v.view(torch.uint8))


# ---------------------------------------------------------------- the debug build
@pytest.mark.parametrize("dtype,kv", KV)
def test_debug_build_gives_the_same_bits(dtype, kv):
    def everything():
        x = _appended(dtype, kv, 128, 16, [3, 40], [7, 0])
        res = [x["qo"], x["ko"], *x["caches"], *(s for s in x["scales"] if s is not None)]
        for f in _calls(dtype, kv, 4):
            res += f()
        torch.cuda.synchronize()
        return res

    a = everything()
    with kda.using_library(kda.load_debug_library()):
        b = everything()
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_debug_build_reports_rows_behind_the_end(monkeypatch):
    for dtype in (BF16, FP32):
        q, k, v, cu = _packed([100, 40], 4, 2, 128, dtype, 7)
        d = [x.cuda() for x in (q, k, v)]
        want, _ = kda.attn_prefill(*d, cu)
        monkeypatch.setenv("KDA_DEBUG_CLIP_TOKENS", "1")
        out = torch.full_like(want, math.nan)
        with kda.using_library(kda.load_debug_library()), pytest.raises(kda.KDAError) as e:
            kda.attn_prefill(*d, cu, out=out)
        assert e.value.code == kda.STATUS_CODES["KDA_ERR_BOUNDS"] and "token row index 139" in str(e.value)
        assert torch.isnan(out[139].float()).all() and torch.equal(out[:139], want[:139])
        monkeypatch.delenv("KDA_DEBUG_CLIP_TOKENS")
