"""Plain float64 forms of the grouped gated delta rule and of the batch plan,
for the tests: the definitions, token by token and request by request."""
from __future__ import annotations

import numpy as np
import torch

EPS32 = 2.0 ** -24     # half a step of fp32, relative
EPS16 = 2.0 ** -8      # half a step of bf16


def tol_state(length, dtype):
    """Relative error (2-norm) a state may have after `length` tokens: about
    eight fp32 roundings a token, adding up as a random walk; the bf16 path also
    carries three operands of its products as two bf16 terms (2^-17 each)."""
    return 8 * np.sqrt(length + 1) * EPS32 + (3 * 2.0 ** -17 if dtype == torch.bfloat16 else 0.0)


def tol_out(length, dtype):
    """Relative error (2-norm) of outputs: bf16 outputs are rounded once, after
    products whose state and masked score operands are rounded to bf16 (three
    roundings of at most half a step each)."""
    return 3 * EPS16 if dtype == torch.bfloat16 else 2 * tol_state(length, dtype)


def rel(x, ref):
    x, ref = np.asarray(x, np.float64), np.asarray(ref, np.float64)
    assert x.shape == ref.shape
    assert np.isfinite(x).all()
    n = np.linalg.norm(ref)
    return float(np.linalg.norm(x - ref) / n) if n else float(np.linalg.norm(x))


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def unit(x):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)


def step(S, q, k, v, g, beta):
    """One token: S [Hv, Dk, Dv], q, k [Hk, Dk], v [Hv, Dv], g, beta [Hv]."""
    rep = v.shape[0] // q.shape[0]
    qh, kh = np.repeat(unit(q), rep, 0), np.repeat(unit(k), rep, 0)
    S = np.where(np.isneginf(g)[:, None, None], 0.0, S * np.exp(g)[:, None, None])
    u = beta[:, None] * (v - np.einsum("hkv,hk->hv", S, kh))
    S = S + kh[:, :, None] * u[:, None, :]
    return S, np.einsum("hkv,hk->hv", S, qh)


def prefill(q, k, v, g, beta, init, lens, stride=0):
    """(out, final states, checkpoints) of packed sequences."""
    q, k, v, g, beta = (f64(x) for x in (q, k, v, g, beta))
    Hv, Dk, Dv = v.shape[1], q.shape[2], v.shape[2]
    out, finals, ckpts, t = np.zeros((sum(lens), Hv, Dv)), [], [], 0
    for n, L in enumerate(lens):
        S = np.zeros((Hv, Dk, Dv)) if init is None or init[n] is None else np.asarray(init[n], np.float64)
        for i in range(L):
            S, out[t] = step(S, q[t], k[t], v[t], g[t], beta[t])
            t += 1
            if stride and (i + 1) % stride == 0:
                ckpts.append(S)
        finals.append(S)
    return out, np.stack(finals), np.stack(ckpts) if ckpts else np.zeros((0, Hv, Dk, Dv))


def inputs(T, Hk, Hv, Dk, Dv, dtype, seed, decay="layer"):
    """Token inputs on the CPU: silu(normal) q, k, v and the gates of a layer."""
    gen = torch.Generator().manual_seed(seed)
    silu = torch.nn.functional.silu
    q, k, v = (silu(torch.randn(T, h, d, generator=gen)).to(dtype) for h, d in ((Hk, Dk), (Hk, Dk), (Hv, Dv)))
    if decay == "layer":
        A = 1 + 15 * torch.rand(Hv, generator=gen)
        g = -A * torch.nn.functional.softplus(torch.randn(T, Hv, generator=gen) - 4)
    else:
        g = torch.full((T, Hv), float(decay))
    return q, k, v, g, torch.sigmoid(torch.randn(T, Hv, generator=gen))


def plan(lens, past, resume, slots, free, head, T, stride, cap, table):
    """The batch plan, request by request; returns a dict of int lists (the table a 2-D list, or None)."""
    N = len(lens)
    past = past or [0] * N
    resume = resume or [-1] * N
    status = 0
    if any(x < 0 for x in lens) or any(x < 0 for x in past) or sum(max(x, 0) for x in lens) > T or not 0 <= head <= len(free):
        status = -1
    past = [max(x, 0) for x in past]
    cu = [0]
    total = 0
    for x in lens:
        total += max(x, 0)
        cu.append(min(total, T))
    L = [cu[n + 1] - cu[n] for n in range(N)]
    if any(past[n] + L[n] > 2 ** 31 - 1 for n in range(N)):
        status = -1
    pos = min(max(head, 0), len(free))
    short = False
    out_slots, init = [], []
    for n in range(N):
        s = slots[n]
        if s < 0 and L[n] > 0:
            if pos < len(free):
                s, pos = free[pos], pos + 1
            else:
                s, short = -1, True
        out_slots.append(s)
        init.append(resume[n] if resume[n] >= 0 else max(slots[n], -1) if past[n] > 0 else -1)
    off, ckpt = [0], []
    table = [list(r) for r in table] if table is not None else None
    for n in range(N):
        due = L[n] // stride if stride else 0
        off.append(off[-1] + due)
        for j in range(due):
            slot = -1
            if len(ckpt) < cap and past[n] % stride == 0 and (table is None or past[n] // stride + j < len(table[n])):
                if pos < len(free):
                    slot, pos = free[pos], pos + 1
                    if table is not None:
                        table[n][past[n] // stride + j] = slot
                else:
                    short = True
            if len(ckpt) < cap:
                ckpt.append(slot)
    if off[-1] > cap:
        short = True
    ckpt += [-1] * (cap - len(ckpt))
    ids, posn = [-1] * T, [-1] * T
    for n in range(N):
        for i in range(L[n]):
            ids[cu[n] + i], posn[cu[n] + i] = n, min(past[n] + i, 2 ** 31 - 1)
    return dict(cu_seqlens=cu, init_slots=init, state_slots=out_slots, ckpt_offsets=off, ckpt_slots=ckpt, seq_ids=ids,
                positions=posn, free_head=[pos], status=status if status else -4 if short else 0, table=table)
