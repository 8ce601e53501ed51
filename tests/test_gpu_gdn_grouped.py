"""Grouped gated delta rule (prefill, decode) against the plain float64 form."""
import numpy as np
import pytest
import torch

import gdn_reference as ref
from gdn_reference import EPS16, f64, rel, tol_out, tol_state
from linear_attention_serving_k1_gb300 import kda

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
SHAPES = [(BF16, 2, 4, 128, 128), (BF16, 1, 3, 128, 192), (BF16, 3, 3, 64, 64), (BF16, 1, 2, 64, 256), (BF16, 2, 2, 128, 512),
          (FP32, 2, 4, 128, 128), (FP32, 1, 2, 64, 64), (FP32, 2, 2, 64, 192)]


def _dev(*xs):
    return [None if x is None else x.cuda().contiguous() for x in xs]


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _init(n, Hv, Dk, Dv, seed=5, scale=0.3):
    return scale * torch.randn(n, Hv, Dk, Dv, generator=torch.Generator().manual_seed(seed))


def _check(out, final, want, lens, dtype):
    L = max(list(lens) + [1])
    o, s = f64(out), f64(final)
    assert rel(o, want[0]) <= tol_out(L, dtype)
    assert rel(s, want[1]) <= tol_state(L, dtype)
    if o.size:
        # no single value further off than its roundings: its own, and those of its row's terms
        rms = np.sqrt(np.mean(want[0] ** 2))
        bound = (EPS16 * np.abs(want[0]) + 8 * EPS16 * rms) if dtype == BF16 else 40 * tol_out(L, dtype) * rms
        assert (np.abs(o - want[0]) <= bound + 1e-30).all()


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", SHAPES)
@pytest.mark.parametrize("lens", [[1], [63, 64, 65], [0, 1, 0, 200, 15, 16, 17, 0]])
def test_prefill(dtype, Hk, Hv, Dk, Dv, lens):
    x = ref.inputs(sum(lens), Hk, Hv, Dk, Dv, dtype, seed=len(lens))
    s0 = _init(len(lens), Hv, Dk, Dv)
    out, final, _ = kda.gdn_prefill(*_dev(*x, s0), _cu(lens))
    _check(out, final, ref.prefill(*x, s0.numpy(), lens), lens, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("decay", [0.0, -1e-3, -0.5, -3.0, -40.0, -np.inf, "resets"])
def test_decays_of_any_size(dtype, decay):
    """No decay, slow, strong (a chunk far below the fp32 range), and states cleared outright."""
    lens = [150, 40]
    x = list(ref.inputs(sum(lens), 1, 2, 128, 128, dtype, seed=3, decay=-0.1 if decay == "resets" else decay))
    if decay == "resets":
        x[3][[0, 5, 63, 64, 100, 149, 150, 170]] = -np.inf
    s0 = _init(2, 2, 128, 128)
    out, final, _ = kda.gdn_prefill(*_dev(*x, s0), _cu(lens))
    _check(out, final, ref.prefill(*x, s0.numpy(), lens), lens, dtype)


@pytest.mark.parametrize("decay", [-1.3, -1.45, -1.5, -1.6])
def test_decays_where_blocks_turn_strong(decay):
    """Both sides of the decay up to which a block of 16 tokens is scaled by its end, and chunks of both kinds in turn."""
    lens = [64, 200]
    x = list(ref.inputs(sum(lens), 1, 2, 128, 64, BF16, seed=31, decay=decay))
    x[3][100:164] *= 1.2
    s0 = _init(2, 2, 128, 64)
    out, final, _ = kda.gdn_prefill(*_dev(*x, s0), _cu(lens))
    _check(out, final, ref.prefill(*x, s0.numpy(), lens), lens, BF16)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_long_sequence(dtype):
    """Many chunks: errors of the carried state do not add up beyond the fp32 roundings."""
    lens = [1500]
    x = list(ref.inputs(1500, 1, 1, 128, 128, dtype, seed=9, decay=-2e-3))
    out, final, _ = kda.gdn_prefill(*_dev(*x), None, _cu(lens))
    _check(out, final, ref.prefill(*x, None, lens), lens, dtype)


def test_equal_lengths_without_offsets_and_zero_state():
    x = ref.inputs(3 * 70, 2, 4, 128, 128, BF16, seed=4)
    out, final, _ = kda.gdn_prefill(*_dev(*x), num_seqs=3)
    _check(out, final, ref.prefill(*x, None, [70] * 3), [70] * 3, BF16)
    out2, none, _ = kda.gdn_prefill(*_dev(*x), num_seqs=3, want_final=False)
    assert none is None and torch.equal(out, out2)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_special_rows(dtype):
    """Zero keys and queries, beta of 0 and beyond 1, equal keys."""
    T = 130
    q, k, v, g, beta = ref.inputs(T, 1, 2, 128, 128, dtype, seed=8)
    k[10:20] = 0
    q[30:33] = 0
    k[64:100] = k[64]
    beta[40:50] = 0
    beta[70:75] = 1.7
    s0 = _init(1, 2, 128, 128)
    out, final, _ = kda.gdn_prefill(*_dev(q, k, v, g, beta, s0), _cu([T]))
    _check(out, final, ref.prefill(q, k, v, g, beta, s0.numpy(), [T]), [T], dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_padded_batch_reads_and_writes_nothing_behind_the_last_sequence(dtype):
    lens, pad = [70, 3], 50
    T = sum(lens) + pad
    x = list(ref.inputs(T, 1, 2, 128, 128, dtype, seed=6))
    want = ref.prefill(*[y[:sum(lens)] for y in x], None, lens)
    for y in x:
        y[sum(lens):] = float("nan")
    out = torch.full((T, 2, 128), 7.0, dtype=dtype, device="cuda")
    _, final, _ = kda.gdn_prefill(*_dev(*x), None, _cu(lens), out=out)
    _check(out[:sum(lens)], final, want, lens, dtype)
    assert (out[sum(lens):] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_neighbouring_sequences_do_not_meet(dtype):
    """Not a number in one sequence stays in it."""
    lens = [70, 40, 65]
    x = list(ref.inputs(sum(lens), 1, 2, 128, 128, dtype, seed=16))
    good = kda.gdn_prefill(*_dev(*x), None, _cu(lens))
    for y in x[:3]:
        y[70:110] = float("nan")
    out, final, _ = kda.gdn_prefill(*_dev(*x), None, _cu(lens))
    for sl in (slice(0, 70), slice(110, 175)):
        assert torch.equal(out[sl], good[0][sl])
    assert torch.equal(final[[0, 2]], good[1][[0, 2]])
    assert torch.isnan(final[1]).any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("which", [3, 4])
def test_gates_that_are_not_numbers_show(dtype, which):
    """In the state of their head and sequence, and nowhere else."""
    lens = [70, 40, 65]
    x = list(ref.inputs(sum(lens), 1, 2, 128, 128, dtype, seed=16))
    good = kda.gdn_prefill(*_dev(*x), None, _cu(lens))
    x[which][75, 1] = float("nan")
    out, final, _ = kda.gdn_prefill(*_dev(*x), None, _cu(lens))
    assert torch.isnan(final[1, 1]).any() and torch.isnan(out[75:110, 1]).any()
    for sl in (slice(0, 70), slice(110, 175)):
        assert torch.equal(out[sl], good[0][sl])
    assert torch.equal(out[:, 0], good[0][:, 0])
    assert torch.equal(final[[0, 2]], good[1][[0, 2]]) and torch.equal(final[1, 0], good[1][1, 0])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_another_stream_while_the_current_one_is_busy(dtype):
    """What a call on the caller's stream allocates and clears does not wait for, or meet, the current stream's work."""
    T, stride = 192, 64
    x = _dev(*ref.inputs(T, 1, 2, 128, 128, dtype, seed=21))
    want = kda.gdn_prefill(*x, ckpt_stride=stride)
    lens = torch.tensor([100, 92], dtype=torch.int32, device="cuda")
    slots = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(7, 17, dtype=torch.int32, device="cuda")
    plan = kda.plan_batch(lens, slots, total_tokens=T, free_slots=free)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)   # (about 0.1 s; it ends by itself)
    got = kda.gdn_prefill(*x, ckpt_stride=stride, stream=side)
    plan2 = kda.plan_batch(lens, slots, total_tokens=T, free_slots=free, stream=side)
    side.synchronize()
    torch.cuda.synchronize()   # and nothing of the current stream's comes after it
    for a, b in zip((*got, *plan2), (*want, *plan)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", SHAPES[:2] + SHAPES[5:6])
def test_checkpoints_and_resume(dtype, Hk, Hv, Dk, Dv):
    lens, stride = [64, 300, 63, 192], 64
    x = ref.inputs(sum(lens), Hk, Hv, Dk, Dv, dtype, seed=2)
    out, final, ck = kda.gdn_prefill(*_dev(*x), None, _cu(lens), ckpt_stride=stride)
    want = ref.prefill(*x, None, lens, stride)
    _check(out, final, want, lens, dtype)
    assert want[2].shape[0] == 8
    assert rel(f64(ck[:8]), want[2]) <= tol_state(300, dtype)
    # the rest of sequence 1 from its second snapshot: the same bits, since chunks restart on the same tokens
    a, b = 64 + 128, 64 + 300
    o2, f2, _ = kda.gdn_prefill(*_dev(*[y[a:b] for y in x]), ck[2:3].contiguous(), _cu([b - a]))
    assert torch.equal(o2, out[a:b]) and torch.equal(f2[0], final[1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n", [1, 30, 31, 32, 60])
def test_checkpoints_and_malformed_offsets_by_the_number_of_sequences(dtype, n):
    """Calls that read their offsets themselves and calls with a table; snapshots, their overflow, offsets out of order."""
    lens = [[64, 0, 130, 7][i % 4] for i in range(n)]
    T = sum(lens)
    x = _dev(*ref.inputs(T, 1, 1, 64, 64, dtype, seed=n))
    due = sum(L // 64 for L in lens)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda").fill_(255)
    more = dict(workspace=ws, max_seq_len=130)   # (the hint: one pass, no segments)
    ck = torch.full((due, 1, 64, 64), 9.0, device="cuda")
    out, final, _ = kda.gdn_prefill(*x, None, _cu(lens), ckpt_stride=64, ckpts=ck, **more)
    assert kda.prefill_status(ws) == 0
    want = ref.prefill(*[y.cpu() for y in x], None, lens, 64)
    _check(out, final, want, lens, dtype)
    assert rel(f64(ck), want[2]) <= tol_state(130, dtype)
    less = torch.full((due, 1, 64, 64), 9.0, device="cuda")
    kda.gdn_prefill(*x, None, _cu(lens), ckpt_stride=64, ckpts=less, ckpt_capacity=due - 1, **more)
    assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_CKPT_OVERFLOW"]
    assert torch.equal(less[:due - 1], ck[:due - 1]) and (less[due - 1] == 9).all()
    for at, value in ((0, 1), (n, T + 1), (n // 2, -1), (n // 2, T + 5)):
        bad = _cu(lens)
        bad[at] = value
        o = torch.full_like(out, 3.0)
        kda.gdn_prefill(*x, None, bad, out=o, **more)
        assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_INVALID_ARG"], (at, value)
        assert (o == 3).all()
    kda.gdn_prefill(*x, None, _cu(lens), **more)
    assert kda.prefill_status(ws) == 0


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 192)])
@pytest.mark.parametrize("longest,n", [(1, 500), (64, 400), (200, 200)])
def test_many_short_sequences(Dk, Dv, longest, n):
    """Far more sequences than the machine runs at once, empty ones among them, with and without a hint."""
    rng = np.random.default_rng(longest)
    lens = [int(x) for x in rng.integers(0, longest + 1, n)]
    x = ref.inputs(sum(lens), 1, 2, Dk, Dv, BF16, seed=longest)
    s0 = _init(n, 2, Dk, Dv)
    out, final, _ = kda.gdn_prefill(*_dev(*x, s0), _cu(lens))
    _check(out, final, ref.prefill(*x, s0.numpy(), lens), lens, BF16)
    for i, L in enumerate(lens):
        if L == 0:
            assert torch.equal(final[i].cpu(), s0[i])
    out2, final2, _ = kda.gdn_prefill(*_dev(*x, s0), _cu(lens), max_seq_len=longest)
    assert torch.equal(out, out2) and torch.equal(final, final2)


@pytest.mark.parametrize("Dk", [64, 128])
@pytest.mark.parametrize("n", [2, 4, 12])
def test_fp32_in_larger_batches(Dk, n):
    """More columns a warp than a small call has: against the plain form, and the bits of the sequences one by one."""
    Hk, Hv, Dv, stride = 4, 16, 64, 64
    lens = [[70, 3, 0, 129, 17, 64][i % 6] for i in range(n)]
    x = ref.inputs(sum(lens), Hk, Hv, Dk, Dv, FP32, seed=n)
    s0 = _init(n, Hv, Dk, Dv)
    out, final, ck = kda.gdn_prefill(*_dev(*x, s0), _cu(lens), ckpt_stride=stride)
    want = ref.prefill(*x, s0.numpy(), lens, stride)
    _check(out, final, want, lens, FP32)
    assert rel(f64(ck[:len(want[2])]), want[2]) <= tol_state(129, FP32)
    at = 0
    for i, L in enumerate(lens):
        if L:
            o, f, _ = kda.gdn_prefill(*_dev(*[y[at:at + L] for y in x], s0[i:i + 1]))
            assert torch.equal(o, out[at:at + L]) and torch.equal(f[0], final[i])
        at += L


def test_too_few_checkpoint_slots_and_malformed_offsets():
    lens = [200, 130]
    x = _dev(*ref.inputs(330, 1, 2, 128, 128, BF16, seed=2))
    desc = kda.make_gdn_desc(330, 1, 2, 128, 128, 2, kda.DTYPE_BF16, 64, 2)
    ws = torch.empty(kda.gdn_workspace_size(desc), dtype=torch.uint8, device="cuda")
    ck = torch.zeros(3, 2, 128, 128, device="cuda")
    out, final, _ = kda.gdn_prefill(*x, None, _cu(lens), ckpt_stride=64, ckpts=ck, ckpt_capacity=2, workspace=ws)
    assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_CKPT_OVERFLOW"]
    assert kda.prefill_status(ws) == 0
    assert torch.count_nonzero(ck[2]) == 0 and torch.count_nonzero(ck[1]) > 0
    for bad in ([0, 200, 100], [0, 200, 331], [5, 200, 330], [0, -4, 330]):
        fin = torch.full_like(final, 3.0)
        o = torch.full_like(out, 3.0)
        kda.gdn_prefill(*x, None, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=o, final_state=fin, workspace=ws)
        assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_INVALID_ARG"]
        assert (o == 3).all()
    kda.gdn_prefill(*x, None, _cu(lens), workspace=ws)
    assert kda.prefill_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_final_state_over_the_initial_one(dtype):
    lens = [0, 90, 64]
    x = _dev(*ref.inputs(154, 2, 2, 128, 128, dtype, seed=2))
    s0 = _init(3, 2, 128, 128).cuda()
    out, final, _ = kda.gdn_prefill(*x, s0, _cu(lens))
    s = s0.clone()
    out2, _, _ = kda.gdn_prefill(*x, s, _cu(lens), final_state=s)
    assert torch.equal(out, out2) and torch.equal(final, s)
    assert torch.equal(s[0], s0[0])


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", SHAPES[:2] + SHAPES[6:])
def test_pooled_prefill_equals_dense(dtype, Hk, Hv, Dk, Dv):
    lens, stride = [130, 0, 64, 5], 64
    x = _dev(*ref.inputs(sum(lens), Hk, Hv, Dk, Dv, dtype, seed=12))
    pool = _init(12, Hv, Dk, Dv).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    init, fin = torch.tensor([3, 11, -1, 99], **i32), torch.tensor([3, 0, 7, -5], **i32)
    ck = torch.tensor([9, -1, 4], **i32)
    s0 = torch.stack([pool[3], pool[11], torch.zeros_like(pool[0]), torch.zeros_like(pool[0])])
    out, final, cks = kda.gdn_prefill(*x, s0, _cu(lens), ckpt_stride=stride, ckpt_capacity=3)
    p = pool.clone()
    o = kda.gdn_prefill_pooled(*x, p, init, fin, _cu(lens), ckpt_stride=stride, ckpt_slots=ck)
    assert torch.equal(o, out)
    want = pool.clone()
    want[3], want[0], want[7], want[9], want[4] = final[0], final[1], final[2], cks[0], cks[2]
    assert torch.equal(p, want)


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", SHAPES)
@pytest.mark.parametrize("N", [1, 5, 200])
def test_decode(dtype, Hk, Hv, Dk, Dv, N):
    if N == 200 and Dv > 256:
        N = 90
    x = ref.inputs(N, Hk, Hv, Dk, Dv, dtype, seed=N)
    s0 = _init(N, Hv, Dk, Dv)
    S = s0.cuda()
    out = kda.gdn_decode(*_dev(*x), S)
    want = ref.prefill(*x, s0.numpy(), [1] * N)
    _check(out, S, want, [1], dtype)
    assert rel(f64(S), want[1]) <= tol_state(1, FP32)     # no operand is rounded here


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", SHAPES[:3] + SHAPES[5:])
def test_decode_continues_prefill(dtype, Hk, Hv, Dk, Dv):
    x = ref.inputs(70, Hk, Hv, Dk, Dv, dtype, seed=31)
    d = _dev(*x)
    _, S, _ = kda.gdn_prefill(*[y[:67].contiguous() for y in d], num_seqs=1)
    outs = [kda.gdn_decode(*[y[t:t + 1].contiguous() for y in d], S) for t in range(67, 70)]
    want = ref.prefill(*x, None, [70])
    assert rel(f64(S), want[1]) <= tol_state(70, dtype)
    assert rel(f64(torch.cat(outs)), want[0][67:]) <= tol_out(70, dtype)


def test_decode_pool_padding_and_repeated_slots():
    N, Hk, Hv, D = 6, 2, 4, 128
    x = _dev(*ref.inputs(N, Hk, Hv, D, D, BF16, seed=1))
    pool = _init(9, Hv, D, D).cuda()
    slots = torch.tensor([4, -1, 0, 9, 8, 2], dtype=torch.int32, device="cuda")
    valid = [0, 2, 4, 5]
    S = pool[slots[valid].long()].clone()
    want = kda.gdn_decode(*[y[valid].contiguous() for y in x], S)
    p, status = pool.clone(), torch.zeros((), dtype=torch.int32, device="cuda")
    out = kda.gdn_decode(*x, p, slot_ids=slots, status=status)
    assert torch.equal(out[valid], want) and torch.count_nonzero(out[[1, 3]]) == 0
    ref_pool = pool.clone()
    ref_pool[slots[valid].long()] = S
    assert torch.equal(p, ref_pool) and status.item() == 0
    slots[5] = 4
    kda.gdn_decode(*x, p, slot_ids=slots, status=status)
    assert status.item() == kda.STATUS_CODES["KDA_ERR_INVALID_ARG"]


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", SHAPES[:4] + SHAPES[5:6])
@pytest.mark.parametrize("N", [3, 120])
def test_decode_multi_commits_a_prefix(dtype, Hk, Hv, Dk, Dv, N):
    m = 4
    x = ref.inputs(N * m, Hk, Hv, Dk, Dv, dtype, seed=N)
    s0 = _init(N, Hv, Dk, Dv)
    commit = torch.randint(-1, m + 2, (N,), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    want = ref.prefill(*x, s0.numpy(), [m] * N)
    d = [y.reshape(N, m, *y.shape[1:]) for y in _dev(*x)]
    S = s0.cuda()
    out = kda.gdn_decode_multi(*d, S, commit_len=commit.cuda())
    assert rel(f64(out).reshape(want[0].shape), want[0]) <= tol_out(m, dtype)
    for n in range(0, N, 7):
        c = min(max(int(commit[n]), 0), m)
        if c == 0:
            assert torch.equal(S[n].cpu(), s0[n])
        else:
            part = ref.prefill(*[y[n * m:n * m + c] for y in x], s0[n:n + 1].numpy(), [c])
            assert rel(f64(S[n]), part[1][0]) <= tol_state(c, FP32)
    # slots and no commit_len: every token
    pool = torch.cat([s0, s0[:1]]).cuda()
    slots = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda")
    out = kda.gdn_decode_multi(*[y.flip(0).contiguous() for y in d], pool, slot_ids=slots)
    assert rel(f64(out.flip(0)).reshape(want[0].shape), want[0]) <= tol_out(m, dtype)
    assert rel(f64(pool[:N]), want[1]) <= tol_state(m, FP32)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP32, 64)])
def test_agrees_with_the_scalar_gate_prefill(dtype, D):
    """Equal head counts and moderate decays: the per-channel entry point's scalar-gate form computes the same thing."""
    lens = [64, 200, 33]
    x = _dev(*ref.inputs(sum(lens), 3, 3, D, D, dtype, seed=21, decay=-0.05))
    out, final, _ = kda.gdn_prefill(*x, None, _cu(lens))
    out2, final2, _ = kda.prefill(*x, None, _cu(lens))
    assert rel(f64(out), f64(out2)) <= 2e-2 and rel(f64(final), f64(final2)) <= 1e-2


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_other_stream_and_captured_calls(dtype):
    """On a stream of the caller's, and captured: two graphs with workspaces of their own, replayed in turn on new values."""
    lens = [100, 28]
    xs = [_dev(*ref.inputs(128, 1, 2, 128, 128, dtype, seed=s)) for s in (1, 2, 3)]
    s0 = _init(2, 2, 128, 128).cuda()
    want = [kda.gdn_prefill(*x, s0, _cu(lens))[:2] for x in xs]
    cu = _cu(lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a = kda.gdn_prefill(*xs[0], s0, cu)
    b = kda.gdn_prefill(*xs[1], s0, cu, stream=stream)
    stream.synchronize()
    for got, w in ((a, want[0]), (b, want[1])):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    n = kda.gdn_workspace_size(kda.make_gdn_desc(128, 1, 2, 128, 128, 2, kda._dtype_code(xs[0][0])))
    held, graphs = [], []
    for _ in range(2):
        st = dict(x=[y.clone() for y in xs[0]], s=s0.clone(), ws=torch.empty(n, dtype=torch.uint8, device="cuda"),
                  out=torch.empty_like(want[0][0]), fin=torch.empty_like(s0))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.gdn_prefill(*st["x"], st["s"], cu, out=st["out"], final_state=st["fin"], workspace=st["ws"])
            st["dec"] = kda.gdn_decode(*[y[:2] for y in st["x"]], st["fin"])
        held.append(st)
        graphs.append(g)
    for st, x in zip(held, xs[1:]):
        for y, z in zip(st["x"], x):
            y.copy_(z)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for st, w, x in zip(held, want[1:], xs[1:]):
        assert torch.equal(st["out"], w[0])
        fin = w[1].clone()
        dec = kda.gdn_decode(*[y[:2] for y in x], fin)
        assert torch.equal(st["fin"], fin) and torch.equal(st["dec"], dec)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_sequences_and_repeatable(dtype):
    """More chains than the machine holds at once, of very different lengths; two runs give the same bits."""
    gen = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 140, (90,), generator=gen).tolist()
    lens[17] = 400
    x = ref.inputs(sum(lens), 2, 4, 64, 128, dtype, seed=5)
    s0 = _init(len(lens), 4, 64, 128)
    d = _dev(*x, s0)
    out, final, _ = kda.gdn_prefill(*d, _cu(lens))
    out2, final2, _ = kda.gdn_prefill(*d, _cu(lens))
    assert torch.equal(out, out2) and torch.equal(final, final2)
    for n in (0, 17, 40, 89):
        a = sum(lens[:n])
        want = ref.prefill(*[y[a:a + lens[n]] for y in x], s0[n:n + 1].numpy(), lens[n:n + 1])
        _check(out[a:a + lens[n]], final[n:n + 1], want, lens[n:n + 1], dtype)


def test_empty_call():
    z = lambda *s, d=BF16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    s0 = _init(2, 2, 64, 64).cuda()
    out, final, _ = kda.gdn_prefill(z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), z(0, 2, d=FP32), z(0, 2, d=FP32), s0,
                                    _cu([0, 0]))
    assert out.shape == (0, 2, 64) and torch.equal(final, s0)
    out = kda.gdn_decode(z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), z(0, 2, d=FP32), z(0, 2, d=FP32), s0[:0])
    assert out.shape == (0, 2, 64)
