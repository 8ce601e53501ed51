"""The gated delta rule (one decay per token and head, value heads sharing a
query/key head) and the batch plan of the state pool, as measured cases: their
inputs, their plain forms in elementary torch operations, the framework's
calls, and their values in 64 bits from the definition.

Per sequence and value head, S fp32 [Dk, Dv], the query/key head of value head
h being h // (Hv / Hk):

    kh = k / sqrt(|k|^2 + 1e-6),  qh = q / sqrt(|q|^2 + 1e-6)
    S' = exp(g_t) S_{t-1}
    S_t = S' + beta_t kh (v_t - S'^T kh)^T
    o_t = S_t^T qh
"""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 64
MAX_COST = 300_000 * 32 * 128          # tokens x value heads x value columns of the largest prefill
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a test-sized call: two heads, one short sequence, all fp32 (latency)
        dict(name="prefill fp32 T256 H2 D64", op="prefill", dtype="fp32", n=1, lo=256, hi=256, lens_seed=0, hk=2, hv=2,
             dk=64, dv=64, stride=0, pooled=False),
        # one short user turn (latency)
        dict(name="prefill bf16 T100 H16/32", op="prefill", dtype="bf16", n=1, lo=100, hi=100, lens_seed=0, hk=16, hv=32,
             dk=128, dv=128, stride=0, pooled=False),
        # one prompt of 8192 tokens, the head count of the framework's second workload
        dict(name="prefill bf16 T8192 H16/32", op="prefill", dtype="bf16", n=1, lo=8192, hi=8192, lens_seed=0, hk=16,
             hv=32, dk=128, dv=128, stride=0, pooled=False),
        # many ragged prompts of a chat service in a state pool, snapshots every 256 tokens
        dict(name="prefill bf16 48 ragged pooled", op="prefill", dtype="bf16", n=48, lo=1, hi=700, lens_seed=3, hk=8, hv=16,
             dk=128, dv=192, stride=256, pooled=True),
        # the framework's varlen workload: 16 prompts of 1024 to 32768 tokens
        dict(name="prefill bf16 16 x U[1024,32768]", op="prefill", dtype="bf16", n=16, lo=1024, hi=32768, lens_seed=1005,
             hk=32, hv=32, dk=128, dv=128, stride=0, pooled=False),
        # fp32 activations, a few prompts
        dict(name="prefill fp32 4 x 2048", op="prefill", dtype="fp32", n=4, lo=1500, hi=2048, lens_seed=5, hk=8, hv=16,
             dk=128, dv=128, stride=0, pooled=False),
        # one user's next token (latency)
        dict(name="decode bf16 N1 H16/32", op="decode", dtype="bf16", n=1, m=1, hk=16, hv=32, dk=128, dv=128, pooled=False,
             pad=0),
        # the framework's decode workload: 256 sequences, 32 heads
        dict(name="decode bf16 N256 H32", op="decode", dtype="bf16", n=256, m=1, hk=32, hv=32, dk=128, dv=128,
             pooled=False, pad=0),
        # a continuous batch over pool slots, some rows padding
        dict(name="decode bf16 N37 pooled", op="decode", dtype="bf16", n=37, m=1, hk=16, hv=32, dk=128, dv=128, pooled=True,
             pad=3),
        # verification of four drafted tokens, a prefix of each committed
        dict(name="decode bf16 N64 m4", op="decode", dtype="bf16", n=64, m=4, hk=16, hv=32, dk=128, dv=128, pooled=True,
             pad=0),
        # the plan of one decode step of 200 requests (latency)
        dict(name="plan N200 decode step", op="plan", n=200, lo=1, hi=1, lens_seed=1, stride=256, new=0),
        # the plan of a mixed batch of long prompts, snapshots every 256 tokens
        dict(name="plan N64 prompts", op="plan", n=64, lo=1, hi=16384, lens_seed=2, stride=256, new=40),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "prefill", "decode", "decode", "plan"))
    if op == "plan":
        n = _log(rng, 1, 4000)
        hi = max(1, min(_log(rng, 1, 20000), 280_000 // n))
        return dict(op=op, n=n, lo=rng.choice((0, 1)) if hi > 1 else 1, hi=hi, lens_seed=rng.randrange(1 << 20),
                    stride=64 * _log(rng, 1, 64), new=rng.randrange(0, n + 1))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    hk, dk, dv = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((64, 128)), rng.choice((64, 128, 128, 192, 256))
    hv = hk * rng.choice((1, 2, 3, 4) if hk <= 4 else (1, 2))
    if op == "decode":
        n, m = _log(rng, 1, 256), rng.choice((1, 1, 1, 2, 3, 5, 8))
        while n * m * hv * dk * dv > 256 * 32 * 128 * 128:
            n //= 2
        pooled = rng.random() < 0.5
        return dict(op=op, dtype=dtype, n=n, m=m, hk=hk, hv=hv, dk=dk, dv=dv, pooled=pooled,
                    pad=rng.randrange(0, n) if pooled and n > 1 and rng.random() < 0.5 else 0)
    n = _log(rng, 1, 60)
    hi = _log(rng, 1, 30000 if dtype == "bf16" else 5000)
    while n * hi * hv * dv > (MAX_COST if dtype == "bf16" else MAX_COST // 16):
        n, hi = max(1, n - 1), max(1, hi * 3 // 4)
    pooled = rng.random() < 0.4
    return dict(op=op, dtype=dtype, n=n, lo=rng.choice((0, 1, hi)) if n > 1 else hi, hi=hi,
                lens_seed=rng.randrange(1 << 20), hk=hk, hv=hv, dk=dk, dv=dv,
                stride=64 * _log(rng, 1, 128) if pooled else 0, pooled=pooled)


def lengths(c):
    r = random.Random(c["lens_seed"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (_prepare_plan if case["op"] == "plan" else _prepare_decode if case["op"] == "decode" else _prepare_prefill)(
        case, gen)


def _tokens(c, gen, rows):
    """q, k, v after the short convolution's SiLU and the gates of a layer: g = -A softplus(a + bias) with A in
    [1, 16] and softplus(bias) in [0.001, 0.1] for each head, beta a sigmoid."""
    dt, hk, hv = DT[c["dtype"]], c["hk"], c["hv"]
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=gen, device=DEV)  # noqa: E731
    q, k, v = (torch.nn.functional.silu(r(*rows, h, d)).to(dt) for h, d in ((hk, c["dk"]), (hk, c["dk"]), (hv, c["dv"])))
    dt0 = torch.exp(math.log(1e-3) + u(hv) * (math.log(0.1) - math.log(1e-3)))
    bias = dt0 + torch.log(-torch.expm1(-dt0))
    g = -(1 + 15 * u(hv)) * torch.nn.functional.softplus(r(*rows, hv) + bias)
    return dict(q=q, k=k, v=v, g=g.contiguous(), beta=torch.sigmoid(r(*rows, hv)))


def _prepare_prefill(c, gen):
    lens = lengths(c)
    n, hv, T = len(lens), c["hv"], sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    s = dict(case=c, lens=lens, cu=cu, **_tokens(c, gen, (T,)))
    if c["pooled"]:
        due = sum(x // c["stride"] for x in lens)
        slots = 2 * n + due
        order = torch.randperm(slots, generator=gen, device=DEV).to(torch.int32)
        s["pool"] = 0.01 * torch.randn(slots, hv, c["dk"], c["dv"], generator=gen, device=DEV)
        s["init"], s["final"], s["ckpt"] = (x.contiguous() for x in (order[:n], order[n:2 * n], order[2 * n:]))
        s["init"][n // 2] = -1          # one request starts from zeros
    else:
        s["s0"] = 0.01 * torch.randn(n, hv, c["dk"], c["dv"], generator=gen, device=DEV)
    return s


def _prepare_decode(c, gen):
    n, m = c["n"], c["m"]
    s = dict(case=c, **_tokens(c, gen, (n, m) if m > 1 else (n,)))
    slots = n + 5 if c["pooled"] else n
    s["state"] = 0.01 * torch.randn(slots, c["hv"], c["dk"], c["dv"], generator=gen, device=DEV)
    s["slots"] = None
    if c["pooled"]:
        s["slots"] = torch.randperm(slots, generator=gen, device=DEV)[:n].to(torch.int32)
        if c["pad"]:
            s["slots"][n - c["pad"]:] = -1
    s["commit"] = torch.randint(0, m + 1, (n,), generator=gen, device=DEV, dtype=torch.int32) if m > 1 else None
    return s


def _prepare_plan(c, gen):
    lens = lengths(c)
    n, T, stride = c["n"], sum(lens), c["stride"]
    due = sum(x // stride for x in lens)
    past = torch.randint(0, 20, (n,), generator=gen, device=DEV, dtype=torch.int32)
    past = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.7, past * stride, past * stride + 7)
    slots = torch.randperm(n, generator=gen, device=DEV).to(torch.int32)
    new = torch.randperm(n, generator=gen, device=DEV)[:c["new"]]
    past[new], slots[new] = 0, -1
    resume = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    some = torch.rand(n, generator=gen, device=DEV) < 0.2
    resume[some] = torch.randint(n, 2 * n, (n,), generator=gen, device=DEV, dtype=torch.int32)[some]
    cols = 20 + max(lens) // stride + 1
    free = (2 * n + torch.randperm(n + due + 8, generator=gen, device=DEV)).to(torch.int32)
    return dict(case=c, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), past=past.to(torch.int32), slots=slots,
                resume=resume, free=free, head=torch.full((1,), 3, dtype=torch.int32, device=DEV),
                table=torch.full((n, cols), -1, dtype=torch.int32, device=DEV), T=T + 13, cap=due + 2)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return (_plan_plain if op == "plan" else _decode_plain if op == "decode" else _prefill_plain)(state)


def _own(op, s):
    from linear_attention_serving_k1_gb300 import kda
    c = s["case"]
    if op == "plan":
        p = kda.plan_batch(s["lens"], s["slots"], total_tokens=s["T"], past=s["past"], resume_slots=s["resume"],
                           ckpt_stride=c["stride"], ckpt_capacity=s["cap"], free_slots=s["free"], free_head=s["head"],
                           snap_table=s["table"])
        return dict(p._asdict(), snap_table=s["table"])
    x = [s[name] for name in ("q", "k", "v", "g", "beta")]
    if op == "decode":
        if c["m"] > 1:
            out = kda.gdn_decode_multi(*x, s["state"], commit_len=s["commit"], slot_ids=s["slots"])
        else:
            out = kda.gdn_decode(*x, s["state"], slot_ids=s["slots"])
        return dict(out=out, state=s["state"])
    if c["pooled"]:
        out = kda.gdn_prefill_pooled(*x, s["pool"], s["init"], s["final"], s["cu"], ckpt_stride=c["stride"],
                                     ckpt_slots=s["ckpt"], max_seq_len=max(s["lens"]))
        return dict(out=out, pool=s["pool"])
    out, final, _ = kda.gdn_prefill(*x, s["s0"], s["cu"], max_seq_len=max(s["lens"]))
    return dict(out=out, final=final)


# ---------------------------------------------------------------- plain forms
def _unit(x):
    x = x.float()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _prefill_plain(s):
    """The recurrence of whole chunks of 64 tokens: with b the running sum of g inside a chunk and
    A = strict-lower(beta_i kh_i.kh_j e^(b_i - b_j)), the chunk's corrections are U = (I + A)^-1 beta (V - e^b K S),
    its outputs e^b Q S + lower(qh_i.kh_j e^(b_i - b_j)) U and its last state e^(b_C) S + K^T e^(b_C - b) U."""
    c, lens = s["case"], s["lens"]
    hk, hv, dk, dv, n = c["hk"], c["hv"], c["dk"], c["dv"], len(lens)
    rep, nc = hv // hk, [-(-x // CHUNK) for x in lens]
    T, total = sum(lens), sum(nc)
    first = [0]
    for x in nc:
        first.append(first[-1] + x)
    start = torch.tensor(first[:-1], device=DEV)
    # rows of every chunk: token, and whether it is inside its sequence
    count = torch.tensor(nc, device=DEV)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), count, output_size=total)
    local = torch.arange(total, device=DEV) - start[seq]
    row = s["cu"].long()[seq][:, None] + local[:, None] * CHUNK + torch.arange(CHUNK, device=DEV)
    there = row < s["cu"].long()[seq + 1][:, None]
    row = torch.where(there, row, torch.full_like(row, T))
    pad = lambda x: torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:], dtype=torch.float32)])  # noqa: E731
    qh = pad(_unit(s["q"]))[row].permute(0, 2, 1, 3)       # [chunks, Hk, 64, Dk]
    kh = pad(_unit(s["k"]))[row].permute(0, 2, 1, 3)
    v = pad(s["v"])[row].permute(0, 2, 1, 3)               # [chunks, Hv, 64, Dv]
    beta = pad(s["beta"])[row].permute(0, 2, 1)            # [chunks, Hv, 64]
    b = torch.cumsum(pad(s["g"])[row].permute(0, 2, 1).double(), -1)   # sums of decays, and their differences
    low = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp(torch.where(low, b[..., :, None] - b[..., None, :], -torch.inf).float())
    eb, el, ec = torch.exp(b).float(), torch.exp(b[..., -1:] - b).float(), torch.exp(b[..., -1]).float()
    share = lambda x: x.repeat_interleave(rep, 1)  # noqa: E731
    A = share(kh @ kh.transpose(-1, -2)) * decay * beta[..., None]
    P = share(qh @ kh.transpose(-1, -2)) * decay
    del decay
    X = torch.eye(CHUNK, device=DEV).expand_as(A)          # (I + A)^-1 of blocks of 1, 2, 4, .. rows
    i = torch.arange(CHUNK, device=DEV)
    for size in (1, 2, 4, 8, 16, 32):
        half = (i[:, None] // size % 2 == 1) & (i[:, None] // size - 1 == i[None, :] // size)
        X = X - X @ torch.where(half, A, torch.zeros((), device=DEV)) @ X
    del A
    qh, kh = share(qh), share(kh)
    out = torch.zeros(T + 1, hv, dv, device=DEV, dtype=s["q"].dtype)
    if c["pooled"]:
        pool, init = s["pool"], s["init"].long()
        S = torch.where((init >= 0)[:, None, None, None], pool[init.clamp(min=0)], torch.zeros((), device=DEV))
        per = [0]
        for x in lens:
            per.append(per[-1] + x // c["stride"])
    else:
        S = s["s0"].clone()
    for step in range(max(nc)):                            # all sequences that have this chunk, at once
        act = [i for i in range(n) if nc[i] > step]
        whole = len(act) == n
        a = torch.tensor(act, device=DEV)
        at = start[a] + step
        K, St = kh[at], S if whole else S[a]
        U = X[at] @ (beta[at][..., None] * (v[at] - eb[at][..., None] * (K @ St)))
        o = eb[at][..., None] * (qh[at] @ St) + P[at] @ U
        St = ec[at][..., None, None] * St + K.transpose(-1, -2) @ (el[at][..., None] * U)
        out[row[at]] = o.permute(0, 2, 1, 3).to(out.dtype)
        if whole:
            S = St
        else:
            S[a] = St
        if c["pooled"] and (step + 1) * CHUNK % c["stride"] == 0:
            done = [i for i in act if lens[i] >= (step + 1) * CHUNK]
            if done:
                j = torch.tensor([per[i] + (step + 1) * CHUNK // c["stride"] - 1 for i in done], device=DEV)
                pool[s["ckpt"].long()[j]] = S[torch.tensor(done, device=DEV)]
    if c["pooled"]:
        pool[s["final"].long()] = S
        return dict(out=out[:T], pool=pool)
    return dict(out=out[:T], final=S)


def _decode_plain(s):
    c, n, m = s["case"], s["case"]["n"], s["case"]["m"]
    rep = c["hv"] // c["hk"]
    q, k, v, g, beta = (s[x].reshape(n, m, *s[x].shape[2 if m > 1 else 1:]) for x in ("q", "k", "v", "g", "beta"))
    qh, kh = _unit(q).repeat_interleave(rep, 2), _unit(k).repeat_interleave(rep, 2)
    there = torch.ones(n, dtype=torch.bool, device=DEV) if s["slots"] is None else s["slots"] >= 0
    at = torch.arange(n, device=DEV) if s["slots"] is None else s["slots"].long().clamp(min=0)
    S = s["state"][at] if s["slots"] is not None else s["state"]
    keep = S
    outs = []
    for t in range(m):
        kt = kh[:, t, :, :, None]
        S = S * torch.exp(g[:, t])[..., None, None]
        u = v[:, t].float() - (S * kt).sum(-2)
        S = S + kt * (beta[:, t, :, None] * u)[..., None, :]
        outs.append((S * qh[:, t, :, :, None]).sum(-2))
        if m > 1:
            keep = torch.where((s["commit"] == t + 1)[:, None, None, None], S, keep)
    out = torch.stack(outs, 1) * there[:, None, None, None]
    S = keep if m > 1 else S
    if s["slots"] is None:
        s["state"].copy_(S)
    elif not c["pad"]:
        s["state"][at] = S
    else:                                                  # padding rows write to a row behind the pool
        big = torch.cat([s["state"], S.new_zeros(1, *S.shape[1:])])
        big[torch.where(there, at, torch.full_like(at, s["state"].shape[0]))] = S
        s["state"].copy_(big[:-1])
    out = out.to(s["q"].dtype)
    return dict(out=out if m > 1 else out[:, 0], state=s["state"])


def _plan_plain(s):
    """The batch plan: token offsets, the slot each request starts from and ends in, slots of the snapshots that fall
    due, and each token's request and position. Free slots go to requests without one first, in order, then to
    snapshots of requests whose past is a whole number of strides, in order."""
    c, T, cap = s["case"], s["T"], s["cap"]
    n, stride, i32 = c["n"], c["stride"], torch.int32
    lens, past = s["lens"].long(), s["past"].long()
    zero = lens.new_zeros(1)
    cu = torch.cat([zero, lens.cumsum(0)])
    want = (s["slots"] < 0) & (lens > 0)
    nth = want.long().cumsum(0) - 1
    head, nfree = s["head"].long(), s["free"].numel()
    free = torch.cat([s["free"].long(), zero - 1])
    place = torch.where(want & (head + nth < nfree), head + nth, nfree)
    final = torch.where(want, free[place], s["slots"].long())
    base = (head + want.sum()).clamp(max=nfree)
    due = lens // stride
    off = torch.cat([zero, due.cumsum(0)])
    e = torch.arange(cap, device=DEV)
    live = e < off[-1]
    mark = torch.zeros(cap + 1, dtype=torch.int64, device=DEV)
    mark.index_add_(0, off[1:-1].clamp(max=cap), torch.ones(n - 1, dtype=torch.int64, device=DEV))
    owner = mark.cumsum(0)[:cap]
    col = past[owner] // stride + e - off[owner]
    fit = live & (past[owner] % stride == 0) & (col < s["table"].shape[1])
    rank = base + fit.long().cumsum(0) - 1
    got = fit & (rank < nfree)
    ckpt = torch.where(got, free[torch.where(got, rank, nfree)], -1)
    width = s["table"].shape[1]
    flat = torch.cat([s["table"].reshape(-1), zero.to(i32)])
    flat[torch.where(got, owner * width + col, n * width)] = ckpt.to(i32)
    s["table"].copy_(flat[:-1].reshape(n, width))
    head_out = (base + fit.sum()).clamp(max=nfree)
    init = torch.where(s["resume"] >= 0, s["resume"].long(), torch.where(past > 0, s["slots"].long().clamp(min=-1), -1))
    t = torch.arange(T, device=DEV)
    mark = torch.zeros(T + 1, dtype=torch.int64, device=DEV)
    mark.index_add_(0, cu[1:-1].clamp(max=T), torch.ones(n - 1, dtype=torch.int64, device=DEV))
    ids = mark.cumsum(0)[:T]
    live = t < cu[-1]
    pos = torch.where(live, past[ids] + t - cu[ids], -1)
    return dict(cu_seqlens=cu.to(i32), init_slots=init.to(i32), state_slots=final.to(i32), ckpt_offsets=off.to(i32),
                ckpt_slots=ckpt.to(i32), seq_ids=torch.where(live, ids, -1).to(i32), positions=pos.to(i32),
                free_head=head_out.to(i32), snap_table=s["table"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "plan":
        lens = lengths(c)
        n, due = c["n"], sum(x // c["stride"] for x in lens)
        return {"bytes": 4.0 * (6 * n + 2 * (sum(lens) + 13) + 3 * due), "flops": 0.0}
    es = 2 if c["dtype"] == "bf16" else 4
    hk, hv, dk, dv = c["hk"], c["hv"], c["dk"], c["dv"]
    block = 4.0 * hv * dk * dv
    if c["op"] == "decode":
        T, states = c["n"] * c["m"], 2 * (c["n"] - c["pad"]) * block
    else:
        lens = lengths(c)
        T = sum(lens)
        states = (2 * c["n"] + (sum(x // c["stride"] for x in lens) if c["pooled"] else 0)) * block
    return {"bytes": T * (2.0 * hk * dk * es + 2.0 * hv * dv * es + 8.0 * hv) + states, "flops": 7.0 * dk * dv * hv * T}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None
    s, c = prepare(case, seed), case
    f = torch.float64
    rep = c["hv"] // c["hk"]

    def step(S, q, k, v, g, beta):
        """One token of the recurrence for a batch [N, H, ...]."""
        q, k = q.to(f), k.to(f)
        q = (q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(rep, 1)
        k = (k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(rep, 1)
        S = S * g.to(f).exp()[..., None, None]
        miss = v.to(f) - torch.einsum("nhkv,nhk->nhv", S, k)
        S = S + torch.einsum("nhk,nhv->nhkv", beta.to(f)[..., None] * k, miss)
        return S, torch.einsum("nhkv,nhk->nhv", S, q)

    x = [s[name] for name in ("q", "k", "v", "g", "beta")]
    if c["op"] == "decode":
        n, m = c["n"], c["m"]
        rows = [i for i in range(n)] if s["slots"] is None else [i for i, p in enumerate(s["slots"].tolist()) if p >= 0]
        at = torch.tensor(rows if s["slots"] is None else [s["slots"].tolist()[i] for i in rows], device=DEV)
        rows = torch.tensor(rows, device=DEV)
        x = [y.reshape(n, m, *y.shape[2 if m > 1 else 1:])[rows] for y in x]
        state = s["state"].to(f)
        S = state[at]
        out = torch.zeros(n, m, c["hv"], c["dv"], dtype=f, device=DEV)
        upto = torch.full((n,), m, device=DEV) if s["commit"] is None else s["commit"]
        for t in range(m):
            S, out[rows, t] = step(S, *(y[:, t] for y in x))
            now = upto[rows] == t + 1
            state[at[now]] = S[now]
        return dict(out=out if m > 1 else out[:, 0], state=state)
    lens = s["lens"]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    if max(lens) * (30e-6 + sum(lens) / max(max(lens), 1) * c["hv"] * c["dk"] * c["dv"] * 64 / 4e12) > 15:
        return None
    cu = s["cu"].tolist()
    if c["pooled"]:
        pool = s["pool"].to(f)
        init = s["init"].tolist()
        first = [0]
        for n_ in lens:
            first.append(first[-1] + n_ // c["stride"])
        S = torch.stack([pool[init[i]] if init[i] >= 0 else torch.zeros_like(pool[0]) for i in order])
        ckpt, final = s["ckpt"].tolist(), s["final"].tolist()
    else:
        S = s["s0"].to(f)[torch.tensor(order, device=DEV)]
    out = torch.zeros(sum(lens), c["hv"], c["dv"], dtype=f, device=DEV)
    begin = torch.tensor([cu[i] for i in order], device=DEV)
    live = len(order)
    for t in range(max(lens)):
        while live and lens[order[live - 1]] <= t:
            live -= 1
        r = begin[:live] + t
        S[:live], out[r] = step(S[:live], *(y[r] for y in x))
        if c["pooled"] and (t + 1) % c["stride"] == 0:
            for j in range(live):
                pool[ckpt[first[order[j]] + (t + 1) // c["stride"] - 1]] = S[j]
    if c["pooled"]:
        for j, i in enumerate(order):
            pool[final[i]] = S[j]
        return dict(out=out, pool=pool)
    back = torch.empty_like(S)
    back[torch.tensor(order, device=DEV)] = S
    return dict(out=out, final=back)
