"""The attention layers that a model interleaves with its linear-attention layers, as measured cases: rotating queries and
keys and writing keys and values into a paged cache, causal attention of packed prompts, attention of new tokens over the
cache (prompts behind a cached past, and single or drafted tokens). Their inputs, their plain forms in elementary torch
operations, the framework's calls, and their values in 64 bits from the definition.

Query head h reads key/value head h // (Hq / Hkv). A query at position p sees the keys 0 .. p of its sequence:

    s_j = q . k_j / sqrt(D),  m = max s_j,  l = sum e^(s_j - m),  o = sum e^(s_j - m) v_j / l,  lse = m + ln l

A cache is [pages, Hkv, page, D]; position p of sequence n lies in page table[n, p // page] at place p % page. An e4m3
cache has one scale per token and head, the smallest power of two s with max |x| <= 448 s.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
MOST_SCORES = 1 << 30                     # scores of one block of a plain form
MOST_FLOPS = {"bf16": 6e12, "fp32": 1e11}   # of a drawn prefill
MOST_CACHE = 1 << 20                      # tokens in a drawn cache, times heads / 8


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token in one layer (latency)
        dict(name="append bf16 N1 H32/8", op="append", dtype="bf16", kv="bf16", n=1, lo=1, hi=1, past=4000, lens_seed=0,
             hq=32, hkv=8, d=128, page=64, rot=128, inter=False, factor=1.0, pad=0),
        # one prompt's 8192 tokens behind 24576 others, an e4m3 cache, frequencies scaled for long contexts
        dict(name="append e4m3 T8192 H32/8", op="append", dtype="bf16", kv="e4m3", n=1, lo=8192, hi=8192, past=24576,
             lens_seed=0, hq=32, hkv=8, d=128, page=64, rot=128, inter=False, factor=8.0, pad=0),
        # a ragged batch in fp32, half of each head rotated in interleaved pairs, padding rows behind it
        dict(name="append fp32 37 ragged", op="append", dtype="fp32", kv="fp32", n=37, lo=1, hi=150, past=2000, lens_seed=2,
             hq=16, hkv=4, d=128, page=16, rot=64, inter=True, factor=1.0, pad=11),
        # a test-sized prompt: two heads, all fp32 (latency)
        dict(name="prefill fp32 T256 H2 D64", op="prefill", dtype="fp32", n=1, lo=256, hi=256, lens_seed=0, hq=2, hkv=2,
             d=64),
        # one prompt of 8192 tokens, the head count of the framework's second workload
        dict(name="prefill bf16 T8192 H32/8", op="prefill", dtype="bf16", n=1, lo=8192, hi=8192, lens_seed=0, hq=32, hkv=8,
             d=128),
        # many ragged prompts of a chat service
        dict(name="prefill bf16 48 ragged D64", op="prefill", dtype="bf16", n=48, lo=1, hi=700, lens_seed=3, hq=16, hkv=4,
             d=64),
        # long documents of the lengths of the framework's varlen workload
        dict(name="prefill bf16 4 x U[1024,32768]", op="prefill", dtype="bf16", n=4, lo=1024, hi=32768, lens_seed=12, hq=32,
             hkv=8, d=128),
        # prompts that resume from a prefix cache
        dict(name="paged bf16 12 ragged", op="paged", dtype="bf16", kv="bf16", n=12, lo=1, hi=900, past=8192, lens_seed=4,
             hq=32, hkv=8, d=128, page=64),
        # one short turn behind a past of the framework's longest prompt
        dict(name="paged e4m3 T100 past 131072", op="paged", dtype="bf16", kv="e4m3", n=1, lo=100, hi=100, past=-131072,
             lens_seed=0, hq=32, hkv=8, d=128, page=64),
        # one user's next token behind a long document (latency)
        dict(name="decode bf16 N1 L32768", op="decode", dtype="bf16", kv="bf16", n=1, m=1, lo=32768, hi=32768, lens_seed=0,
             hq=32, hkv=8, d=128, page=64),
        # a full batch of ragged conversations
        dict(name="decode bf16 N256 ragged", op="decode", dtype="bf16", kv="bf16", n=256, m=1, lo=1, hi=8192, lens_seed=7,
             hq=32, hkv=8, d=128, page=64),
        # verification of four drafted tokens over an e4m3 cache
        dict(name="decode e4m3 N64 m4", op="decode", dtype="bf16", kv="e4m3", n=64, m=4, lo=4, hi=16384, lens_seed=8, hq=32,
             hkv=8, d=128, page=32),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("append", "append", "prefill", "prefill", "paged", "decode", "decode"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    hkv, d = rng.choice((1, 2, 3, 4, 8, 8, 16)), rng.choice((64, 128, 128))
    c = dict(op=op, dtype=dtype, hq=hkv * rng.choice((1, 2, 3, 4, 5, 8) if hkv <= 4 else (1, 2, 3, 4)), hkv=hkv, d=d,
             lens_seed=rng.randrange(1 << 20))
    if op != "prefill":
        c.update(kv=rng.choice(("bf16", "e4m3")) if dtype == "bf16" else "fp32", page=rng.choice((16, 32, 64, 64, 128)))
    if op == "decode":
        n, hi = _log(rng, 1, 256), _log(rng, 1, 40000)
        while n * hi * hkv * d > MOST_CACHE * 8 * 128 * 2:
            n, hi = max(1, n * 3 // 4), max(1, hi * 3 // 4)
        m = rng.choice((1, 1, 1, 2, 3, 5, 8))
        return dict(c, n=n, m=m, hi=max(hi, m), lo=min(max(hi, m), rng.choice((0, 1, hi))))
    n, hi = _log(rng, 1, 60), _log(rng, 1, 20000 if dtype == "bf16" else 2500)
    past = 0 if op == "prefill" or rng.random() < 0.2 else _log(rng, 1, 30000)
    while (n * hi * (hi / 2 + past) * c["hq"] * d * 4 > MOST_FLOPS[dtype] or n * (hi + past) * hkv * d > MOST_CACHE * 8 * 128
           or n * hi * c["hq"] * d > 1 << 28):
        n, hi, past = max(1, n * 3 // 4), max(1, hi * 3 // 4), past * 3 // 4
    c.update(n=n, hi=hi, lo=rng.choice((0, 1, hi)) if n > 1 else hi)
    if op == "append":
        c.update(rot=rng.choice((d, d, d // 2, d // 4, 6)), inter=rng.random() < 0.5, factor=rng.choice((1.0, 1.0, 4.0, 32.0)),
                 pad=rng.randrange(0, 20))
    return c if op == "prefill" else dict(c, past=past)


def lengths(c):
    """New tokens of each sequence, and cached tokens before them."""
    r = random.Random(c["lens_seed"])
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]
    lens[c["n"] // 2] = c["hi"]
    past = c.get("past", 0)
    if c["op"] == "decode":               # `lens` counts the new tokens in
        return [c["m"]] * c["n"], [x - c["m"] for x in lens]
    return lens, [-past if past < 0 else r.randint(0, past) for _ in lens]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c, dt = case, DT[case["dtype"]]
    lens, past = lengths(c)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    T, hq, hkv, d = sum(lens) + c.get("pad", 0), c["hq"], c["hkv"], c["d"]
    s = dict(case=c, lens=lens, past=past, cu=torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV))
    if c["op"] == "decode":
        s["q"] = (2 * r(c["n"], c["m"], hq, d)).to(dt)
    else:
        s["q"] = (2 * r(T, hq, d)).to(dt)
    if c["op"] in ("append", "prefill"):
        # a few channels far above the others, as keys have them
        s["k"], s["v"] = (r(T, hkv, d) * (1 + 4 * (torch.arange(d, device=DEV) % 29 == 3))).to(dt), r(T, hkv, d).to(dt)
    if c["op"] == "prefill":
        return s
    total = [a + b for a, b in zip(lens, past)]
    _cache(s, gen, [max(0, x) for x in total], c["op"] == "append")
    s["kv_lens"] = torch.tensor([max(0, x) for x in total], dtype=torch.int32, device=DEV)
    if c["op"] == "append":
        i32 = dict(dtype=torch.int32, device=DEV)
        n, first = torch.tensor(lens, device=DEV), s["cu"][:-1].long()
        ids = torch.repeat_interleave(torch.arange(c["n"], device=DEV), n)
        pos = torch.arange(sum(lens), device=DEV) - first[ids] + torch.tensor(past, device=DEV)[ids]
        none = torch.full((c["pad"],), -1, **i32)
        s["seq_ids"], s["positions"] = torch.cat([ids.to(torch.int32), none]), torch.cat([pos.to(torch.int32), none])
        s["inv_freq"], s["rope_scale"] = _frequencies(c["rot"], c["factor"])
        s["q_out"] = torch.zeros_like(s["q"])
    return s


def _frequencies(rot, factor, base=500000.0, original=8192, fast=32.0, slow=1.0):
    """Frequencies base^(-2i / rot), those of fewer than `slow` turns over the original context divided by `factor`, those
    of more than `fast` kept, a ramp between; and the factor on cosine and sine that goes with them."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    if factor == 1.0:
        return f.float().to(DEV), 1.0
    turns = original * f / (2 * math.pi)
    ramp = ((torch.log(turns) - math.log(slow)) / (math.log(fast) - math.log(slow))).clamp(0, 1)
    return (f * (ramp + (1 - ramp) / factor)).float().to(DEV), 0.1 * math.log(factor) + 1.0


def _cache(s, gen, total, empty):
    """Pages in a random order, a table with -1 behind each sequence's last page."""
    c = s["case"]
    page, hkv, d = c["page"], c["hkv"], c["d"]
    need = [-(-x // page) for x in total]
    width = max(need) + 1
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    n = torch.tensor(need, device=DEV)
    there = torch.arange(width, device=DEV)[None, :] < n[:, None]
    table = torch.full((c["n"], width), -1, dtype=torch.int32, device=DEV)
    table[there] = order[:sum(need)]
    s["table"] = table
    shape = (pages, hkv, page, d)
    for name in ("k", "v"):
        if c["kv"] == "e4m3":
            codes = torch.empty(shape, dtype=F8, device=DEV)
            for a in range(0, pages, 4096):                # (in parts: normal values take four times the bytes)
                part = codes[a:a + 4096]
                part.copy_((90 * (not empty) * torch.randn(part.shape, generator=gen, device=DEV)).clamp(-448, 448))
            e = torch.randint(-8, -5, shape[:3], generator=gen, device=DEV)
            s[name + "_cache"], s[name + "_scale"] = codes, torch.ldexp(torch.ones((), device=DEV), e if not empty else 0 * e)
        else:
            x = torch.zeros(shape, dtype=DT[c["kv"]], device=DEV)
            s[name + "_cache"] = x if empty else x.normal_(generator=gen)
            s[name + "_scale"] = None


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return (_append_plain if op == "append" else _prefill_plain if op == "prefill" else _paged_plain)(state)


def _own(op, s):
    from linear_attention_serving_k1_gb300 import kda
    c = s["case"]
    if op == "append":
        kda.kv_append(s["q"], s["k"], s["v"], s["positions"], seq_ids=s["seq_ids"], page_table=s["table"],
                      k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                      inv_freq=s["inv_freq"], interleaved=c["inter"], rope_scale=s["rope_scale"], q_out=s["q_out"])
        return _written(s)
    if op == "prefill":
        out, lse = kda.attn_prefill(s["q"], s["k"], s["v"], s["cu"], max_seq_len=max(s["lens"]), want_lse=True)
        return dict(out=out, lse=lse)
    cache = (s["k_cache"], s["v_cache"], s["table"], s["kv_lens"])
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], want_lse=True)
    if op == "paged":
        out, lse = kda.attn_prefill_paged(s["q"], *cache, s["cu"], max_seq_len=max(s["lens"]), **scales)
    elif c["m"] > 1:
        out, lse = kda.attn_decode_multi(s["q"], *cache, **scales)
    else:
        out, lse = kda.attn_decode(s["q"][:, 0], *cache, **scales)
        out, lse = out[:, None], lse[:, None]
    return dict(out=out, lse=lse)


def _written(s):
    """Queries and the cache; e4m3 values as the tensor that holds them, with their scales."""
    names = ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")
    return {n: s[n] for n in names if s[n] is not None}


# ---------------------------------------------------------------- plain forms
def _turned(x, angle_cos, angle_sin, inter):
    rot = 2 * angle_cos.shape[-1]
    head, rest = x[..., :rot], x[..., rot:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
    co, si = angle_cos[:, None], angle_sin[:, None]
    a, b = a * co - b * si, a * si + b * co
    head = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([head, rest], -1)


def _append_plain(s):
    c = s["case"]
    there = s["positions"] >= 0
    at = there.nonzero().flatten()
    pos, ids = s["positions"].long()[at], s["seq_ids"].long()[at]
    angle = pos.double()[:, None] * s["inv_freq"].double()
    co, si = (torch.cos(angle) * s["rope_scale"]).float(), (torch.sin(angle) * s["rope_scale"]).float()
    s["q_out"][at] = _turned(s["q"][at].float(), co, si, c["inter"]).to(s["q"].dtype)
    page, place = s["table"].long()[ids, pos // c["page"]], pos % c["page"]
    for name, x in (("k", _turned(s["k"][at].float(), co, si, c["inter"])), ("v", s["v"][at].float())):
        if c["kv"] == "e4m3":
            x, scale = _eight(x)
            s[name + "_scale"][page, :, place] = scale.float()
        s[name + "_cache"].view(torch.uint8 if c["kv"] == "e4m3" else x.dtype if c["kv"] == "fp32" else torch.bfloat16)[
            page, :, place] = x.view(torch.uint8) if c["kv"] == "e4m3" else x.to(DT[c["kv"]])
    return _written(s)


def _eight(x):
    """e4m3 values and the power of two that they are multiplied by."""
    m, e = torch.frexp(x.abs().amax(-1))
    scale = torch.ldexp(torch.ones_like(m), torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126))
    return (x / scale[..., None]).to(F8), scale


def _attend(q, k, v, limit, scale):
    """q [B, Hkv, rows, D], k, v [B, Hkv, keys, D], limit [B, 1, rows, 1]: keys that a row sees."""
    sc = (q @ k.transpose(-1, -2)) * scale
    j = torch.arange(k.shape[2], device=DEV)
    sc = torch.where(j < limit, sc, -torch.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isinf(m), 0.0, m))
    del sc
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    return o, lse


def _prefill_plain(s):
    c, lens = s["case"], s["lens"]
    most = max(lens)
    row = s["cu"].long()[:-1, None] + torch.arange(most, device=DEV)
    row = torch.where(row < s["cu"].long()[1:, None], row, sum(lens))     # [N, longest], a row of zeros behind
    pad = lambda x: torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:], dtype=torch.float32)])  # noqa: E731
    k, v = pad(s["k"])[row].transpose(1, 2), pad(s["v"])[row].transpose(1, 2)
    return _blocks(s, k, v, row, torch.zeros(c["n"], dtype=torch.long, device=DEV))


def _blocks(s, k, v, row, past):
    """Blocks of query rows of all sequences at once, so many that their scores fit."""
    c = s["case"]
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    G, T, most = hq // hkv, s["q"].shape[0], row.shape[1]
    out = torch.zeros(T + 1, hq, d, device=DEV, dtype=s["q"].dtype)
    lse = torch.full((T + 1, hq), -torch.inf, device=DEV)
    q = torch.cat([s["q"], s["q"].new_zeros(1, hq, d)])
    step = max(1, min(most, MOST_SCORES // (n * hq * k.shape[2])))
    ahead = max(s["past"])
    for a in range(0, most, step):
        r = row[:, a:a + step]
        w = r.shape[1]
        x = q[r].float().reshape(n, w, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, G * w, d)
        limit = past[:, None] + torch.arange(a, a + w, device=DEV) + 1
        upto = min(k.shape[2], ahead + a + w)
        o, l = _attend(x, k[:, :, :upto], v[:, :, :upto], limit.repeat(1, G)[:, None, :, None], d ** -0.5)
        out[r] = o.reshape(n, hkv, G, w, d).permute(0, 3, 1, 2, 4).reshape(n, w, hq, d).to(out.dtype)
        lse[r] = l.reshape(n, hkv, G, w).permute(0, 3, 1, 2).reshape(n, w, hq)
    return dict(out=out[:T], lse=lse[:T])


def _read(s, name):
    """[N, Hkv, longest, D] of the cache, zeros behind each sequence's end."""
    c = s["case"]
    most = max(1, int(max(a + b for a, b in zip(s["lens"], s["past"]))))
    pages = s["table"].long()[:, :-(-most // c["page"])]
    x = s[name + "_cache"][pages.clamp(min=0)].float()      # [N, pages, Hkv, page, D]
    if c["kv"] == "e4m3":
        x = x * s[name + "_scale"][pages.clamp(min=0)][..., None]
    x = x.transpose(1, 2).flatten(2, 3)
    there = torch.arange(x.shape[2], device=DEV) < s["kv_lens"][:, None]
    return x.mul_(there[:, None, :, None])


def _paged_plain(s):
    c, n = s["case"], s["case"]["n"]
    k, v = _read(s, "k"), _read(s, "v")
    past = torch.tensor(s["past"], device=DEV)
    if c["op"] == "paged":
        row = s["cu"].long()[:-1, None] + torch.arange(max(s["lens"]), device=DEV)
        return _blocks(s, k, v, torch.where(row < s["cu"].long()[1:, None], row, sum(s["lens"])), past)
    m, hq, hkv, d = c["m"], c["hq"], c["hkv"], c["d"]
    q = s["q"].float().reshape(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    limit = (past[:, None] + torch.arange(m, device=DEV) + 1).repeat(1, hq // hkv)
    o, l = _attend(q, k, v, limit[:, None, :, None], d ** -0.5)
    o = o.reshape(n, hkv, hq // hkv, m, d).permute(0, 3, 1, 2, 4).reshape(n, m, hq, d)
    return dict(out=o.to(s["q"].dtype), lse=l.reshape(n, hkv, hq // hkv, m).permute(0, 3, 1, 2).reshape(n, m, hq))


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    lens, past = lengths(c)
    es, T, hq, hkv, d = 2.0 if c["dtype"] == "bf16" else 4.0, sum(lens), c["hq"], c["hkv"], c["d"]
    kv = 2 * hkv * (d + 4.0 if c.get("kv") == "e4m3" else d * es)       # bytes of a token in the cache
    if c["op"] == "append":
        return {"bytes": T * (es * d * (2 * hq + 2 * hkv) + kv + 8.0), "flops": 3.0 * T * (hq + hkv) * c["rot"]}
    seen = sum(x * p + x * (x + 1) / 2 for x, p in zip(lens, past) if x > 0 and x + p > 0)
    flops = 4.0 * d * hq * max(seen, 0.0)
    if c["op"] == "prefill":
        return {"bytes": T * es * d * (2 * hq + 2 * hkv) + 4.0 * T * hq, "flops": flops}
    read = sum(max(0, x + p) for x, p in zip(lens, past) if x > 0)
    return {"bytes": T * (2 * es * d + 4.0) * hq + read * kv, "flops": flops}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = case
    lens, past = lengths(c)
    f = torch.float64
    if c["op"] == "append":
        return _append_exact(c, prepare(case, seed), f)
    if sum(4.0 * c["d"] * c["hq"] * x * (max(p, 0) + x) for x, p in zip(lens, past)) > 6e12:
        return None
    s = prepare(case, seed)
    hq, hkv, d, m = c["hq"], c["hkv"], c["d"], c.get("m", 1)
    q = s["q"].reshape(-1, hq, d)
    out = torch.zeros(q.shape, dtype=f, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=f, device=DEV)
    first = 0
    for n, (L, P) in enumerate(zip(lens, past)):            # one sequence after another, and one head group
        if L and P + L > 0:
            for g in range(hkv):
                if c["op"] == "prefill":
                    K, V = s["k"][first:first + L, g].to(f), s["v"][first:first + L, g].to(f)
                else:
                    rows = s["table"][n, :-(-(P + L) // c["page"])].long()
                    K, V = (s[x + "_cache"][rows, g].to(f) * (1.0 if s[x + "_scale"] is None else
                                                              s[x + "_scale"][rows, g].to(f)[..., None]) for x in "kv")
                    K, V = K.reshape(-1, d)[:P + L], V.reshape(-1, d)[:P + L]
                for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                    for a in range(0, L, 4096):
                        at = torch.arange(a, min(L, a + 4096), device=DEV)
                        z = q[first + at, h].to(f) @ K.T / math.sqrt(d)
                        z.masked_fill_(torch.arange(P + L, device=DEV)[None, :] > (at + P)[:, None], -math.inf)
                        total = torch.logsumexp(z, 1)
                        w = torch.exp(z - total.clamp(min=-1e300)[:, None])
                        out[first + at, h], lse[first + at, h] = w @ V, total
        first += L
    return dict(out=out.reshape(s["q"].shape), lse=lse.reshape(s["q"].shape[:-1]))


def _append_exact(c, s, f):
    """Each pair as a complex number times e^(i angle)."""
    w = {n: x.to(f) for n, x in _written(s).items()}
    rot, page = c["rot"], c["page"]
    pairs = torch.arange(rot).reshape(-1, 2) if c["inter"] else torch.arange(rot).reshape(2, -1).T
    first, second = pairs[:, 0].to(DEV), pairs[:, 1].to(DEV)

    def turn(x, pos):
        z = torch.complex(x[..., first], x[..., second])
        z = z * torch.polar(torch.full((), s["rope_scale"], dtype=f, device=DEV), pos.to(f) * s["inv_freq"].to(f))[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    live = s["seq_ids"] >= 0
    pos, ids = s["positions"][live][:, None], s["seq_ids"][live].long()
    w["q_out"][live] = turn(s["q"][live].to(f), pos)
    pg, place = s["table"][ids, pos[:, 0].long() // page].long(), pos[:, 0].long() % page
    for name, x in (("k", turn(s["k"][live].to(f), pos)), ("v", s["v"][live].to(f))):
        if c["kv"] == "e4m3":
            # the smallest power of two that brings the largest to 448 or less; then the nearest e4m3 value: a step is 1/8
            # of the power of two below the value, and at least 2^-9; halves go to the even one
            top = x.abs().amax(-1).clamp(min=1e-300)
            scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-126))
            y = x / scale[..., None]
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            x, w[name + "_scale"][pg, :, place] = torch.round(y / step) * step, scale
        w[name + "_cache"][pg, :, place] = x
    return w
