"""Values that are not finite in the grouped gated delta rule's prefill: they show from
their token on, in the heads and columns that they reach by the formula, and nowhere else."""
import numpy as np
import pytest
import torch

import gdn_reference as ref
from gdn_reference import EPS16, f64, rel, tol_out, tol_state
from linear_attention_serving_k1_gb300 import kda

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _check(dtype, Hk, Hv, Dk, Dv, lens, seed, spoil, **more):
    """spoil(q, k, v, g, beta) puts the values in; the plain form says where they reach."""
    x = ref.inputs(sum(lens), Hk, Hv, Dk, Dv, dtype, seed=seed)
    s0 = 0.3 * torch.randn(len(lens), Hv, Dk, Dv, generator=torch.Generator().manual_seed(seed))
    first, x = x, [y.clone() for y in x]
    spoil(*x)
    # the same call with only the values that are no numbers as they were (-inf is a decay)
    keep = [torch.isfinite(y) | (torch.isneginf(y) if i == 3 else False) for i, y in enumerate(x)]
    clean = [torch.where(m, y, z).cuda() for m, y, z in zip(keep, x, first)]
    with np.errstate(all="ignore"):
        want, wfin, wck = ref.prefill(*x, s0.numpy(), lens, 64)
    assert not np.isfinite(want).all()
    n = len(wck)
    out, fin, ck = kda.gdn_prefill(*[y.cuda() for y in x], s0.cuda(), _cu(lens), ckpt_stride=64, **more)
    good, gfin, gck = kda.gdn_prefill(*clean, s0.cuda(), _cu(lens), ckpt_stride=64, **more)
    L = max(lens)
    for got, w, c, tol in ((out, want, good, tol_out(L, dtype)), (fin, wfin, gfin, tol_state(L, dtype)),
                           (ck[:n], wck, gck[:n], tol_state(L, dtype))):
        ok = np.isfinite(w)
        got = f64(got)
        assert (np.isfinite(got) == ok).all()
        assert rel(got[ok], w[ok]) <= tol
        # (and what no such value reaches is close to the call without them)
        assert rel(got[ok], f64(c)[ok]) <= 2 * tol


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 1, 6, 15, 16, 37, 63, 64, 77, 99])
def test_a_key_reaches_its_value_heads_from_its_token_on(dtype, bad, at):
    def spoil(q, k, v, g, beta):
        k[at, 1, 9] = bad
    _check(dtype, 2, 4, 64, 64, [100, 30], at, spoil)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 2, 15, 16, 45, 63, 64, 97, 99])
def test_a_value_reaches_its_column_from_its_token_on(dtype, bad, at):
    def spoil(q, k, v, g, beta):
        v[at, 1, 100] = bad
    _check(dtype, 1, 2, 128, 192, [100, 30], at, spoil)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("which,bad", [(3, NAN), (4, NAN), (4, INF), (4, -INF)])
@pytest.mark.parametrize("at", [0, 3, 14, 17, 63, 64, 82, 99])
def test_a_gate_reaches_its_head_from_its_token_on(dtype, which, bad, at):
    def spoil(*x):
        x[which][at, 1] = bad
    _check(dtype, 1, 3, 64, 64, [100, 30], at, spoil)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("at", [0, 18, 64, 99])
def test_a_query_reaches_its_own_row(dtype, bad, at):
    def spoil(q, k, v, g, beta):
        q[at, 0, 5] = bad
    _check(dtype, 2, 2, 64, 64, [100, 30], at, spoil)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_several_at_once(dtype):
    """Values of several columns and tokens of a chunk and the next, before and behind a key, beside strong and no decay."""
    def spoil(q, k, v, g, beta):
        for t, h, c, y in ((3, 0, 0, NAN), (40, 0, 0, INF), (20, 0, 63, NAN), (70, 0, 64, -INF), (12, 1, 191, NAN), (90, 1, 5, NAN)):
            v[t, h, c] = y
        k[80, 0, 0] = NAN
        g[30:60] = -40.0
        g[2] = -INF
        v[101:110, 1, 7] = INF
    _check(dtype, 1, 2, 64, 192, [95, 70], 5, spoil)


@pytest.mark.parametrize("which", ["k", "v", "g"])
def test_in_segments(which):
    """Long sequences with few heads: a segment behind the value starts from what it left."""
    def spoil(q, k, v, g, beta):
        if which == "k":
            k[1000, 0, 3] = NAN
        elif which == "v":
            v[1000, 1, 77] = NAN
        else:
            g[1000, 1] = NAN
    _check(BF16, 1, 2, 128, 128, [1500, 100], 8, spoil)


def test_a_huge_key_does_not_reach_earlier_tokens():
    """A key whose squares overflow fp32: tokens before it are as ever."""
    x = list(ref.inputs(60, 1, 1, 64, 64, BF16, seed=2))
    want = ref.prefill(*[y[:30] for y in x], None, [30])[0]
    x[1] = x[1].clone()
    x[1][30] = 3e38
    out, _, _ = kda.gdn_prefill(*[y.cuda() for y in x], None, _cu([60]))
    assert rel(f64(out[:30]), want) <= 3 * EPS16


@pytest.mark.parametrize("longest,n", [(64, 500), (200, 250)])
def test_among_many_short_sequences(longest, n):
    """Chains of one chunk and of none in turn on every SM, values of every third sequence not finite: those show in their
    column from their token on, the rest has the bits of the call without them."""
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, longest + 1, n)]
    x = list(ref.inputs(sum(lens), 1, 2, 64, 192, BF16, seed=n))
    clean = [y.cuda() for y in x]
    out, fin, _ = kda.gdn_prefill(*clean, None, _cu(lens), max_seq_len=longest)
    v, at, where = x[2].clone(), 0, []
    for i, L in enumerate(lens):
        if L and i % 3 == 0:
            t, h, c = int(rng.integers(L)), int(rng.integers(2)), int(rng.integers(192))
            v[at + t, h, c] = (NAN, INF, -INF)[i // 3 % 3]
            where.append((i, at + t, at + L, h, c))
        at += L
    got, gfin, _ = kda.gdn_prefill(*clean[:2], v.cuda(), *clean[3:], None, _cu(lens), max_seq_len=longest)
    out, fin, got, gfin = (f64(y) for y in (out, fin, got, gfin))
    for i, a, b, h, c in where:
        assert np.isnan(got[a:b, h, c]).all() and np.isnan(gfin[i, h, :, c]).all()
        got[a:b, h, c], gfin[i, h, :, c] = out[a:b, h, c], fin[i, h, :, c]
    assert np.array_equal(got, out) and np.array_equal(gfin, fin)
