"""Plain float64 forms of the attention layers, for the tests: rotation, the paged
cache's e4m3 rows, and causal attention over packed or paged keys, with the error
that each element of a result may have."""
from __future__ import annotations

import math

import torch

F64, F8 = torch.float64, torch.float8_e4m3fn
EPS32 = 2.0 ** -24     # half a step of fp32, relative
EPS16 = 2.0 ** -8      # half a step of bf16


def f64(t):
    return t.detach().cpu().to(F64)


# ---------------------------------------------------------------- rotation and cache rows
def rotate(x, pos, inv_freq, interleaved, scale):
    """x [T, H, D] float64, pos [T], inv_freq fp32 [R / 2]."""
    R = 2 * len(inv_freq)
    ang = pos.to(F64)[:, None] * f64(inv_freq)
    co, si = (scale * ang.cos())[:, None], (scale * ang.sin())[:, None]
    i = torch.arange(R // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y = x.clone()
    y[..., ia], y[..., ib] = x[..., ia] * co - x[..., ib] * si, x[..., ia] * si + x[..., ib] * co
    return y


def scale_of(x):
    """The power of two of a row (last dim): the smallest s >= 2^-126 with max |x| <= 448 s."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return torch.where(top.isfinite(), torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, torch.full_like(e, -126))),
                       torch.full_like(top, math.nan))


def codes(x, s):
    """x / s rounded to nearest e4m3, halves to even, as float64."""
    y = x / s[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


# ---------------------------------------------------------------- attention
def attend(q, k, v, first, scale):
    """One sequence: q [L, Hq, D], k, v [S, Hkv, D] float64; query i sees keys 0 .. first + i.  Returns (out, lse, A, d):
    A = sum of p |v| / l per element, d = how much a score's magnitude sums to (sum |q k| scale, the largest)."""
    L, Hq, D = q.shape
    rep = Hq // k.shape[1]
    out, lse, A, d = (torch.zeros(L, Hq, D, dtype=F64), torch.full((L, Hq), -math.inf, dtype=F64), torch.zeros(L, Hq, D, dtype=F64),
                      torch.zeros(L, Hq, dtype=F64))
    for i in range(L):
        n = first + i + 1
        if n <= 0:
            continue
        K, V = k[:n].repeat_interleave(rep, 1), v[:n].repeat_interleave(rep, 1)
        s = torch.einsum("hd,shd->hs", q[i], K) * scale
        m = s.amax(1)
        p = torch.exp(s - m[:, None])
        l = p.sum(1)
        out[i] = torch.einsum("hs,shd->hd", p, V) / l[:, None]
        A[i] = torch.einsum("hs,shd->hd", p, V.abs()) / l[:, None]
        lse[i] = m + torch.log(l)
        d[i] = (torch.einsum("hd,shd->hs", q[i].abs(), K.abs()) * scale).amax(1)
    return out, lse, A, d


def attend_all(q, k, v, lens, past, scale):
    """Packed queries of sequences with lens new tokens behind `past`; k, v: lists of [S, Hkv, D]."""
    parts, t = [], 0
    for n, L in enumerate(lens):
        parts.append(attend(q[t:t + L], k[n], v[n], past[n], scale))
        t += L
    return [torch.cat(x) for x in zip(*parts)]


def tolerance(want, lse, A, d, n, D, dtype):
    """Per element.  A score of D products is off by at most (D / 4 + 8) fp32 roundings of d (blocked sums), a weight by
    twice that relative to l, sums of n terms by 4 sqrt(n) + 8 roundings.  bf16 outputs are rounded once, and the
    weights of the product with V once (a bf16 cache of the framework's tensor-core path): half a step each."""
    ds = (D / 4 + 8) * EPS32 * d
    more = 2 * ds + (4 * math.sqrt(n) + 16) * EPS32
    out = more[..., None] * A + EPS32 * want.abs()
    if dtype == torch.bfloat16:
        out = out + EPS16 * want.abs() + EPS16 * (1 + more[..., None]) * A
    return out + 1e-30, ds + (4 * math.sqrt(n) + 16 + lse.abs().nan_to_num(posinf=0.0)) * EPS32


def check(out, lse, q, k, v, lens, past, scale=None):
    """Compares a call's results on real tensors with the definition (k, v: lists of [S, Hkv, D] float64)."""
    D = q.shape[-1]
    want, wl, A, d = attend_all(f64(q).reshape(-1, *q.shape[-2:]), k, v, lens, past, scale or D ** -0.5)
    tol, tl = tolerance(want, wl, A, d, max([a + b for a, b in zip(lens, past)] + [1]), D, q.dtype)
    got = f64(out).reshape(want.shape)
    err = (got - want).abs()
    assert got.isfinite().all()
    assert (err <= tol).all(), f"output: {float((err / tol).max()):.3g} of the tolerance at {int((err / tol).argmax())}"
    if lse is not None:
        gl = f64(lse).reshape(wl.shape)
        none = torch.isinf(wl)
        assert torch.equal(torch.isneginf(gl), none)
        el = (gl - wl)[~none].abs()
        assert (el <= tl[~none]).all(), f"lse: {float((el / tl[~none]).max()):.3g} of the tolerance"


# ---------------------------------------------------------------- inputs
class Case:
    """A batch over a paged cache: sequences of kv_lens tokens, the last lens[n] of them new; pages in a random order, every
    place of the cache that no sequence holds filled with NaN (e4m3: its scale)."""

    def __init__(self, lens, past, Hq, Hkv, D, page, dtype, kv="same", seed=0, spare=2, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.past, self.page = list(lens), list(past), page
        total = [max(0, a + b) for a, b in zip(lens, past)]
        need = [-(-x // page) for x in total]
        pages, self.cols = sum(need) + spare, max(need + [1]) + 1
        order = torch.randperm(pages, generator=g)
        self.q = (2 * torch.randn(sum(lens), Hq, D, generator=g)).to(dtype)
        self.k = [(torch.randn(x, Hkv, D, generator=g) * (1 + 3 * (torch.arange(D) % 29 == 3))).to(dtype) for x in total]
        self.v = [torch.randn(x, Hkv, D, generator=g).to(dtype) for x in total]
        table = torch.full((len(lens), self.cols), -1, dtype=torch.int32)
        caches = [torch.full((pages, Hkv, page, D), math.nan, dtype=dtype) for _ in range(2)]
        scales = [torch.full((pages, Hkv, page), math.nan) for _ in range(2)]
        at = 0
        for n, x in enumerate(total):
            table[n, :need[n]] = order[at:at + need[n]].to(torch.int32)
            for c, rows in zip(caches, (self.k[n], self.v[n])):
                for j in range(x):
                    c[order[at + j // page], :, j % page] = rows[j]
            at += need[n]
        if kv == "e4m3":
            for i in range(2):
                x = caches[i].to(F64)
                live = x.isfinite().all(-1)
                s = torch.where(live, scale_of(x.nan_to_num(0.0)), torch.full((), math.nan, dtype=F64))
                scales[i] = s.float()
                y = codes(x.nan_to_num(0.0), torch.where(live, s, torch.ones((), dtype=F64)))
                caches[i] = torch.where(live[..., None], y, torch.full((), 448.0, dtype=F64)).float().to(F8)
            # what attention is defined on: code times scale
            self.k, self.v = ([self._read(caches[i], scales[i], table[n], x) for n, x in enumerate(total)] for i in range(2))
        else:
            scales = [None, None]
            self.k, self.v = [f64(x) for x in self.k], [f64(x) for x in self.v]
        to = lambda x: None if x is None else x.to(device)  # noqa: E731
        self.cache = tuple(to(x) for x in (*caches, table, torch.tensor(total, dtype=torch.int32)))
        self.scales = dict(k_scale=to(scales[0]), v_scale=to(scales[1]))
        self.qd = to(self.q)
        self.cu = torch.tensor([0] + self.lens).cumsum(0).to(torch.int32).to(device)

    def _read(self, cache, scale, table, x):
        j = torch.arange(x)
        pg = table[j // self.page].long()
        return cache.float()[pg, :, j % self.page].to(F64) * scale[pg, :, j % self.page].to(F64)[..., None]

    def check(self, out, lse):
        check(out, lse, self.q, self.k, self.v, self.lens, self.past)
