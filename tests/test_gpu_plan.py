"""The batch plan against its plain form, and the plan, prefill and decode of a
serving loop run together."""
import random

import numpy as np
import pytest
import torch

import gdn_reference as ref
from gdn_reference import f64, rel, tol_out, tol_state
from linear_attention_serving_k1_gb300 import kda

pytestmark = pytest.mark.gpu


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32).reshape(-1 if not x or not isinstance(x[0], list) else (len(x), -1)).cuda()


def _compare(lens, past, resume, slots, free, head, T, stride, cap, table):
    want = ref.plan(lens, past, resume, slots, free, head, T, stride, cap, table)
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    tab = _i32(table)
    p = kda.plan_batch(_i32(lens), _i32(slots), total_tokens=T, past=_i32(past), resume_slots=_i32(resume),
                       ckpt_stride=stride, ckpt_capacity=cap, free_slots=_i32(free), free_head=_i32([head]),
                       snap_table=tab, status=status)
    for name, got in p._asdict().items():
        assert got.tolist() == want[name], name
    assert status.item() == want["status"]
    if table is not None:
        assert tab.tolist() == want["table"]
    return p


@pytest.mark.parametrize("N,hi,stride", [(1, 1, 64), (3, 200, 64), (40, 1, 64), (200, 300, 128), (257, 40, 0), (1500, 30, 64),
                                         (16384, 3, 64)])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan(N, hi, stride, seed):
    r = random.Random(100 * N + seed)
    lens = [r.randint(0, hi) for _ in range(N)]
    past = [r.choice((0, 64, 128, 640, 7)) for _ in range(N)]
    resume = [r.choice((-1, -1, r.randint(0, 9999))) for _ in range(N)]
    slots = [r.choice((-1, r.randint(0, 9999), -7)) for _ in range(N)]
    T = sum(lens) + r.choice((0, 1, 77))
    due = sum(x // stride for x in lens) if stride else 0
    free = r.sample(range(10000, 60000), N + due + 5)
    if seed:   # too few free slots, too few columns
        free = free[:max(1, len(free) // 3)]
    table = [[-9] * (3 if seed else 30)] * N if N < 2000 else None
    _compare(lens, past, resume, slots, free, r.randint(0, 2) if len(free) > 2 else 0, T, stride, due + 3 if not seed else due // 2,
             table)


def test_plan_refusals_seen_on_the_device():
    base = dict(past=None, resume=None, slots=[-1, 4, -1], free=[8, 9], head=0, stride=64, cap=2, table=None)
    _compare([5, -3, 2], T=9, **base)                                   # a negative length counts as none
    _compare([5, 3, 2], T=9, **base)                                    # more tokens than rows
    _compare([5, 3, 2], T=10, **dict(base, head=7))                     # free_head beyond the list
    _compare([5, 3, 2], T=10, **dict(base, head=-1))
    _compare([5, 3, 2], T=10, **dict(base, past=[-2, 2 ** 31 - 2, 0]))  # a position beyond int32
    _compare([5, 3, 2], T=10, **dict(base, free=[]))                    # no free slot at all
    _compare([0, 0, 0], T=0, **base)
    _compare([2 ** 31 - 1] * 3, T=130, **base)                          # a sum beyond int32


def test_plan_in_place_and_captured():
    """state_slots and free_head advanced in place, the call replayed as a graph on new lengths."""
    N, T, stride = 5, 400, 64
    lens, slots, head = _i32([10, 20, 30, 0, 130]), _i32([-1, 2, -1, -1, -1]), _i32([1])
    free, table = _i32(list(range(100, 120))), torch.full((N, 4), -1, dtype=torch.int32, device="cuda")
    past = _i32([0, 6, 0, 0, 0])
    first = kda.plan_batch(lens, slots, total_tokens=T, past=past, ckpt_stride=stride, ckpt_capacity=4, free_slots=free,
                           free_head=head, snap_table=table.clone())
    out = kda.BatchPlan(*(torch.empty_like(x) for x in first))._replace(state_slots=slots, free_head=head)
    start = [x.clone() for x in (slots, head)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.plan_batch(lens, slots, total_tokens=T, past=past, ckpt_stride=stride, ckpt_capacity=4, free_slots=free,
                       free_head=head, snap_table=table, out=out)
    for x, y in zip((slots, head), start):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, first):
        assert torch.equal(a, b)
    assert slots.tolist() == [101, 2, 102, -1, 103] and head.item() == 6
    assert table[4].tolist() == [104, 105, -1, -1]
    lens.copy_(_i32([1, 1, 1, 1, 1]))
    g.replay()
    torch.cuda.synchronize()
    assert slots.tolist() == [101, 2, 102, 106, 103] and head.item() == 7
    assert out.cu_seqlens.tolist() == [0, 1, 2, 3, 4, 5] and out.seq_ids[5:].eq(-1).all()


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", [(torch.bfloat16, 1, 2, 128, 128), (torch.float32, 1, 2, 64, 64)])
def test_serving_loop(dtype, Hk, Hv, Dk, Dv):
    """Three requests prefilled in a padded batch, one continued and one resumed from a snapshot of another, then decoded:
    every table comes from the plan, none from the host."""
    stride, pool_slots = 64, 24
    pool = torch.full((pool_slots, Hv, Dk, Dv), 5.0, device="cuda")
    free, head = _i32(list(range(pool_slots - 1, -1, -1))), _i32([0])
    slots, past, table = _i32([-1, -1, -1, -1]), _i32([0, 0, 0, 0]), torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    seqs = [ref.inputs(260, Hk, Hv, Dk, Dv, dtype, seed=s) for s in range(3)]
    taken = [0, 0, 0]

    def batch(lens, T, resume=None):
        """Packs the next lens[n] tokens of each request into T rows and runs plan and prefill."""
        parts = []
        for n, L in enumerate(lens[:3]):
            parts.append([y[taken[n]:taken[n] + L] for y in seqs[n]])
            taken[n] += L
        x = [torch.cat([p[i] for p in parts]) for i in range(5)]
        x = [torch.cat([y, torch.full((T - y.shape[0], *y.shape[1:]), float("nan"), dtype=y.dtype)]).cuda() for y in x]
        plan = kda.plan_batch(_i32(lens), slots, total_tokens=T, past=past, resume_slots=resume, ckpt_stride=stride,
                              ckpt_capacity=8, free_slots=free, free_head=head, snap_table=table)
        out = kda.gdn_prefill_pooled(*x, pool, plan.init_slots, plan.state_slots, plan.cu_seqlens, ckpt_stride=stride,
                                     ckpt_slots=plan.ckpt_slots)
        slots.copy_(plan.state_slots)
        head.copy_(plan.free_head)
        past.add_(_i32(lens))
        return out

    first = batch([128, 70, 200, 0], 420)
    second = batch([130, 0, 9, 0], 139)
    want = [ref.prefill(*[y[:taken[n]] for y in seqs[n]], None, [taken[n]], stride) for n in range(3)]
    assert rel(f64(first[:128]), want[0][0][:128]) <= tol_out(128, dtype)
    assert rel(f64(first[128:198]), want[1][0]) <= tol_out(70, dtype)
    assert rel(f64(second[:130]), want[0][0][128:]) <= tol_out(258, dtype)
    assert rel(f64(second[130:139]), want[2][0][200:]) <= tol_out(209, dtype)
    # the snapshot table: request 0 after 64..256 tokens (its second prefill starts on the grid), request 2 after 64..192
    for n, count in ((0, 4), (1, 1), (2, 3)):
        ids = table[n].tolist()
        assert all(s >= 0 for s in ids[:count]) and all(s < 0 for s in ids[count:])
        for j in range(count):
            assert rel(f64(pool[ids[j]]), want[n][2][j]) <= tol_state(260, dtype)
    # a fourth request shares the first 128 tokens of request 0: it starts from that snapshot
    tail = [y[128:160] for y in seqs[0]]
    resume = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    resume[3] = table[0, 1]
    past[3] = 128
    plan = kda.plan_batch(_i32([0, 0, 0, 32]), slots, total_tokens=32, past=past, resume_slots=resume, ckpt_stride=stride,
                          free_slots=free, free_head=head, snap_table=table)
    out = kda.gdn_prefill_pooled(*[y.cuda() for y in tail], pool, plan.init_slots, plan.state_slots, plan.cu_seqlens)
    assert rel(f64(out), want[0][0][128:160]) <= tol_out(160, dtype)
    assert plan.positions.tolist() == list(range(128, 160))
    slots.copy_(plan.state_slots)
    # one decode step of requests 1 and 2, the others idle: padding rows
    step = _i32([0, 1, 1, 0])
    ids = torch.where(step > 0, slots, torch.full_like(slots, -1))
    before = pool.clone()
    x = [torch.stack([seqs[n][i][taken[n]] if n in (1, 2) else seqs[0][i][0] for n in (0, 1, 2, 0)]).cuda() for i in range(5)]
    out = kda.gdn_decode(*x, pool, slot_ids=ids)
    for n in (1, 2):
        w = ref.prefill(*[y[:taken[n] + 1] for y in seqs[n]], None, [taken[n] + 1])
        assert rel(f64(out[n]), w[0][-1]) <= tol_out(taken[n], dtype)
        assert rel(f64(pool[slots[n]]), w[1][0]) <= tol_state(taken[n], dtype)
    rest = [i for i in range(pool_slots) if i not in (slots[1].item(), slots[2].item())]
    assert torch.equal(pool[rest], before[rest])
    assert np.all(f64(out[[0, 3]]) == 0)
