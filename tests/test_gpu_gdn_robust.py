"""Grouped gated delta rule beyond the numbers: waits that give up, the debug
build, two calls at once, offsets beyond 32 bits."""
import pytest
import torch

import gdn_reference as ref
from gdn_reference import f64, rel, tol_out, tol_state
from linear_attention_serving_k1_gb300 import kda

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
BOUNDS = kda.STATUS_CODES["KDA_ERR_BOUNDS"]


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _inputs(lens, Hk, Hv, Dk, Dv, dtype, seed):
    x = ref.inputs(sum(lens), Hk, Hv, Dk, Dv, dtype, seed)
    s0 = 0.3 * torch.randn(len(lens), Hv, Dk, Dv, generator=torch.Generator().manual_seed(seed + 1))
    return x, s0, [y.cuda() for y in x], s0.cuda()


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 192)])
def test_waits_give_up_and_the_next_call_is_clean(Dk, Dv):
    """A wait limit of one poll: the call returns, its status says so, and the workspace and GPU are as good as before."""
    lens = [300, 70, 1]
    x, s0, d, s = _inputs(lens, 2, 4, Dk, Dv, BF16, 61)
    desc = kda.make_gdn_desc(sum(lens), 2, 4, Dk, Dv, 3, kda.DTYPE_BF16)
    ws = torch.empty(kda.gdn_workspace_size(desc), dtype=torch.uint8, device="cuda")
    kda.gdn_prefill(*d, s, _cu(lens), workspace=ws, wait_limit=1)
    assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_TIMEOUT"]
    out, final, _ = kda.gdn_prefill(*d, s, _cu(lens), workspace=ws)
    assert kda.prefill_status(ws) == 0
    want = ref.prefill(*x, s0.numpy(), lens)
    assert rel(f64(out), want[0]) <= tol_out(300, BF16) and rel(f64(final), want[1]) <= tol_state(300, BF16)


@pytest.mark.parametrize("dtype,Dk,Dv", [(BF16, 128, 128), (BF16, 64, 192), (FP32, 128, 64)])
def test_debug_build_gives_the_same_bits(dtype, Dk, Dv):
    lens = [1, 64, 130, 0, 200]
    _, _, d, s = _inputs(lens, 2, 4, Dk, Dv, dtype, 62)

    def everything():
        out, final, ck = kda.gdn_prefill(*d, s, _cu(lens), ckpt_stride=64, ckpt_capacity=6)
        pool = torch.cat([s, s])
        slots = torch.tensor([3, 9, -1, 0, 1], dtype=torch.int32, device="cuda")
        po = kda.gdn_prefill_pooled(*d, pool, slots, slots, _cu(lens))
        step = [y[:5].contiguous() for y in d]
        st = final.clone()
        o1 = kda.gdn_decode(*step, st)
        o2 = kda.gdn_decode_multi(*[y[:10].reshape(5, 2, *y.shape[1:]).contiguous() for y in d], st)
        i = torch.arange(5, dtype=torch.int32, device="cuda")
        plan = kda.plan_batch(i * 70, i - 2, total_tokens=800, ckpt_stride=64, ckpt_capacity=9, free_slots=i + 50)
        torch.cuda.synchronize()
        return [out, final, ck, pool, po, o1, o2, st, *plan]

    a = everything()
    with kda.using_library(kda.load_debug_library()):
        b = everything()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_debug_build_reports_rows_behind_the_end(monkeypatch, dtype):
    """The checks take the token buffers to be one row shorter: the last row is skipped and reported."""
    lens = [70, 65]
    T = sum(lens)
    _, _, d, s = _inputs(lens, 1, 2, 128, 128, dtype, 63)
    want, _, _ = kda.gdn_prefill(*d, s, _cu(lens))
    step = [y[:4].contiguous() for y in d]
    st0 = s[:1].repeat(4, 1, 1, 1)
    st_ref = st0.clone()
    dec = kda.gdn_decode(*step, st_ref)
    dbg = kda.load_debug_library()
    monkeypatch.setenv("KDA_DEBUG_CLIP_TOKENS", "1")
    out, st, od = torch.full_like(want, float("nan")), st0.clone(), torch.full_like(dec, float("nan"))
    with kda.using_library(dbg):
        with pytest.raises(kda.KDAError) as e:
            kda.gdn_prefill(*d, s, _cu(lens), out=out)
        assert e.value.code == BOUNDS and f"token row index {T - 1} outside [0, {T - 1})" in str(e.value)
        with pytest.raises(kda.KDAError) as e:
            kda.gdn_decode(*step, st, out=od)
        assert e.value.code == BOUNDS
    assert torch.isnan(out[T - 1].float()).all() and torch.equal(out[:T - 1], want[:T - 1])
    assert torch.isnan(od[3].float()).all() and torch.equal(od[:3], dec[:3])
    assert torch.equal(st[3], st0[3]) and torch.equal(st[:3], st_ref[:3])
    monkeypatch.delenv("KDA_DEBUG_CLIP_TOKENS")
    with kda.using_library(dbg):
        again, _, _ = kda.gdn_prefill(*d, s, _cu(lens))
    assert torch.equal(again, want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_two_calls_at_once(dtype):
    """On two streams, each with its own workspace, many times: the same bits as one after the other."""
    lens = [[500, 20], [64, 333, 90]]
    calls = [_inputs(x, 2, 4, 128, 128, dtype, 70 + i)[2:] for i, x in enumerate(lens)]
    want = [kda.gdn_prefill(*d, s, _cu(x))[:2] for (d, s), x in zip(calls, lens)]
    cu = [_cu(x) for x in lens]
    streams = [torch.cuda.Stream() for _ in lens]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(kda.gdn_prefill(*calls[i][0], calls[i][1], cu[i])[:2])
    torch.cuda.synchronize()
    for i in range(2):
        for o, f in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(f, want[i][1])


def test_rows_and_slots_beyond_32_bits():
    """v and out of more than 2^31 elements, a pool of more than 2^31 floats: the last rows and slots as in small calls."""
    Hk, Hv, Dk, Dv = 1, 32, 64, 256
    lens = [2 ** 31 // (Hv * Dv) + 37, 100]
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k = (torch.randn(T, Hk, Dk, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    v = torch.randn(T, Hv, Dv, generator=gen, device="cuda", dtype=BF16)
    g, beta = -torch.rand(T, Hv, generator=gen, device="cuda"), torch.rand(T, Hv, generator=gen, device="cuda")
    out, final, _ = kda.gdn_prefill(q, k, v, g, beta, None, _cu(lens))
    tail = [y[lens[0]:].clone() for y in (q, k, v, g, beta)]
    out2, final2, _ = kda.gdn_prefill(*tail, num_seqs=1)
    assert torch.equal(out[lens[0]:], out2) and torch.equal(final[1], final2[0])
    out3, final3, _ = kda.gdn_prefill(*[y[:64].clone() for y in (q, k, v, g, beta)], num_seqs=1)
    assert torch.equal(out[:64], out3)
    del v, out
    Hv, Dk, Dv = 32, 128, 512
    slots = 2 ** 31 // (Hv * Dk * Dv) + 3
    pool = torch.zeros(slots, Hv, Dk, Dv, device="cuda")
    pool[-1] = torch.randn(Hv, Dk, Dv, generator=gen, device="cuda")
    x = [y.cuda() for y in ref.inputs(1, 4, Hv, Dk, Dv, BF16, 5)]
    st = pool[-1:].clone()
    o = kda.gdn_decode(*x, st)
    o2 = kda.gdn_decode(*x, pool, slot_ids=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, o2) and torch.equal(pool[-1], st[0]) and torch.count_nonzero(pool[:-1]) == 0


@pytest.mark.parametrize("Hk,Hv,Dk,Dv,lens,hint", [
    (1, 1, 128, 128, [2500], 0), (1, 2, 64, 64, [1999], 0), (1, 3, 128, 192, [1280], 0), (2, 2, 128, 64, [1300, 0, 64, 700], 0),
    (1, 2, 128, 256, [900, 1500, 1], 1500), (1, 1, 64, 128, [1900, 63], 800)])
def test_few_long_chains_in_segments(Hk, Hv, Dk, Dv, lens, hint):
    """Few heads and long sequences run in segments, joined: outputs, states and snapshots as ever, with a length hint that
    is right, absent or too short."""
    x, s0, d, s = _inputs(lens, Hk, Hv, Dk, Dv, BF16, 80 + len(lens))
    stride = 192
    want = ref.prefill(*x, s0.numpy(), lens, stride)
    out, final, ck = kda.gdn_prefill(*d, s, _cu(lens), ckpt_stride=stride, max_seq_len=hint)
    L = max(lens)
    assert rel(f64(out), want[0]) <= tol_out(L, BF16)
    assert rel(f64(final), want[1]) <= tol_state(L, BF16)
    assert rel(f64(ck[:want[2].shape[0]]), want[2]) <= tol_state(L, BF16)
    # through a pool, its final slots the initial ones; twice, the same bits
    ids = torch.randperm(len(lens), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    for _ in range(2):
        pool = torch.empty_like(s)
        pool[ids.long()] = s
        o2 = kda.gdn_prefill_pooled(*d, pool, ids, ids, _cu(lens), max_seq_len=hint)
        assert torch.equal(o2, out) and torch.equal(pool[ids.long()], final)


def test_segments_reset_and_decay():
    """Segments whose transition vanishes (a cleared state) and is nearly the identity (no decay)."""
    for decay in (0.0, -0.5):
        lens = [1600]
        x = list(ref.inputs(1600, 1, 1, 128, 128, BF16, 91, decay=decay))
        x[3][777] = float("-inf")
        out, final, _ = kda.gdn_prefill(*[y.cuda() for y in x], None, _cu(lens))
        want = ref.prefill(*x, None, lens)
        assert rel(f64(out), want[0]) <= tol_out(1600, BF16) and rel(f64(final), want[1]) <= tol_state(1600, BF16)


@pytest.mark.parametrize("lens", [[8192], [8100, 700]])
def test_segments_in_more_rounds_than_one(lens):
    """More segments than the machine runs at once, against the same call in one pass (a hint of short sequences)."""
    _, _, x, s0 = _inputs(lens, 2, 32 // len(lens), 64, 64, BF16, 77)
    whole, cut = (kda.gdn_prefill(*x, s0, _cu(lens), ckpt_stride=256, max_seq_len=hint) for hint in (64, max(lens)))
    n = sum(L // 256 for L in lens)
    # each is within its tolerance of the exact values
    assert rel(f64(cut[0]), f64(whole[0])) <= 2 * tol_out(max(lens), BF16)
    assert rel(f64(cut[1]), f64(whole[1])) <= 2 * tol_state(max(lens), BF16)
    assert rel(f64(cut[2][:n]), f64(whole[2][:n])) <= 2 * tol_state(max(lens), BF16)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n", [3, 5, 31, 40])
def test_offsets_whose_differences_wrap_are_refused(dtype, n):
    """Interior offsets far out of range, whose differences in 32 bits look like lengths: nothing is read or written."""
    T = 330
    x = [y.cuda() for y in ref.inputs(T, 1, 2, 64, 64, dtype, seed=n)]
    s0 = 0.3 * torch.randn(n, 2, 64, 64, generator=torch.Generator().manual_seed(2)).cuda()
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda").fill_(255)
    for far in ([2_000_000_000, -2_000_000_000], [2 ** 31 - 1, -2 ** 31], [2 ** 30, -2 ** 30 - 5], [2 ** 31 - 1, 2 ** 31 - 1],
                [-2 ** 31, -1]):
        cu = torch.tensor([0] + far + [T] * (n - 2), dtype=torch.int32, device="cuda")
        out = torch.full((T, 2, 64), 3.0, dtype=dtype, device="cuda")
        fin = torch.full_like(s0, 3.0)
        kda.gdn_prefill(*x, s0, cu, out=out, final_state=fin, workspace=ws, max_seq_len=T)
        assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_INVALID_ARG"], far
        assert (out == 3).all() and torch.equal(fin, s0)


@pytest.mark.parametrize("first", [0, 64, 200])
def test_every_wait_that_gave_up_is_reported(first):
    """With a limit of one poll and stale words in the workspace, whether the first CTA has work or none: no such call reports
    that all went well, and none hides the report of the next."""
    lens = [first] + [300] * 14
    _, _, d, s = _inputs(lens, 1, 2, 128, 128, BF16, 64)
    cu, n = _cu(lens), kda.gdn_workspace_size(kda.make_gdn_desc(sum(lens), 1, 2, 128, 128, len(lens), kda.DTYPE_BF16, max_seq_len=300))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for stale in (0, 255, 1, 0, 255):
        ws.fill_(stale)
        kda.gdn_prefill(*d, s, cu, workspace=ws, wait_limit=1, max_seq_len=300)
        assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_TIMEOUT"]
    ws.fill_(255)
    out, final, _ = kda.gdn_prefill(*d, s, cu, workspace=ws, max_seq_len=300)
    assert kda.prefill_status(ws) == 0
    again, fin2, _ = kda.gdn_prefill(*d, s, cu, max_seq_len=300)
    assert torch.equal(out, again) and torch.equal(final, fin2)


def test_equal_sequences_are_planned_by_their_own_length():
    """Without offsets every sequence has T / N tokens: the same workspace and the same bits as with that hint."""
    N, L, Hk, Hv, D = 4, 2048, 4, 8, 128
    x = [y.cuda() for y in ref.inputs(N * L, Hk, Hv, D, D, BF16, seed=6)]
    desc = [kda.make_gdn_desc(N * L, Hk, Hv, D, D, N, kda.DTYPE_BF16, max_seq_len=m) for m in (L, 0)]
    n, unknown = (kda.gdn_workspace_size(d) for d in desc)
    assert n < unknown
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out, final, _ = kda.gdn_prefill(*x, num_seqs=N, workspace=ws)
    want = kda.gdn_prefill(*x, None, _cu([L] * N), max_seq_len=L)
    assert torch.equal(out, want[0]) and torch.equal(final, want[1])
    pool = torch.zeros(N, Hv, D, D, device="cuda")
    ids = torch.arange(N, dtype=torch.int32, device="cuda")
    out = kda.gdn_prefill_pooled(*x, pool, None, ids, num_seqs=N, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(pool, want[1])


@pytest.mark.parametrize("dtype,Hk,Hv,Dk,Dv", [(BF16, 2, 4, 128, 128), (FP32, 1, 3, 64, 192), (BF16, 2, 8, 128, 256)])
@pytest.mark.parametrize("N,m", [(7, 4), (60, 3), (7, 1), (5, 2)])
def test_decode_multi_over_a_pool(dtype, Hk, Hv, Dk, Dv, N, m):
    """Padding rows, lengths to commit from none to all and beyond, and slots at once; then a slot named twice."""
    x = ref.inputs(N * m, Hk, Hv, Dk, Dv, dtype, seed=N)
    P = N + 6
    gen = torch.Generator().manual_seed(N)
    pool = 0.3 * torch.randn(P, Hv, Dk, Dv, generator=gen)
    slots = torch.randperm(P, generator=gen)[:N].to(torch.int32)
    slots[1], slots[3], slots[4] = -1, P, 2 ** 31 - 1
    commit = torch.tensor([(i * 2) % (m + 3) - 1 for i in range(N)], dtype=torch.int32)
    d = [y.reshape(N, m, *y.shape[1:]).cuda() for y in x]
    p, status = pool.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kda.gdn_decode_multi(*d, p, commit_len=commit.cuda(), slot_ids=slots.cuda(), status=status)
    assert status.item() == 0
    want = pool.clone()
    for n in range(N):
        s, rows = int(slots[n]), slice(n * m, n * m + m)
        if not 0 <= s < P:
            assert torch.count_nonzero(out[n]) == 0
            continue
        w = ref.prefill(*[y[rows] for y in x], pool[s:s + 1].numpy(), [m])
        assert rel(f64(out[n]), w[0]) <= tol_out(m, dtype)
        c = min(max(int(commit[n]), 0), m)
        if c > 0:
            part = ref.prefill(*[y[n * m:n * m + c] for y in x], pool[s:s + 1].numpy(), [c])
            assert rel(f64(p[s]), part[1][0]) <= tol_state(c, FP32)
            want[s] = p[s].cpu()
    assert torch.equal(p.cpu(), want)      # no other slot was touched
    slots[N - 1] = slots[0]
    kda.gdn_decode_multi(*d, p, slot_ids=slots.cuda(), status=status)
    assert status.item() == kda.STATUS_CODES["KDA_ERR_INVALID_ARG"]


@pytest.mark.parametrize("lens,hint", [([1500, 700], 0), ([1999, 64, 0, 300], 1999)])
def test_segments_over_a_pool_with_snapshots(lens, hint):
    """Initial, final and snapshot slots apart from one another, some left out: the states of the dense call, no other slot
    touched."""
    Hk, Hv, D, stride, n = 1, 2, 128, 128, len(lens)
    x, s0, d, s = _inputs(lens, Hk, Hv, D, D, BF16, 90 + n)
    due = sum(L // stride for L in lens)
    P = 2 * n + due + 5
    desc = kda.make_gdn_desc(sum(lens), Hk, Hv, D, D, n, kda.DTYPE_BF16, stride, due, hint)
    assert kda.gdn_workspace_size(desc) > 4 * n * Hv * D * D      # (segments: states in the workspace)
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(n)).to(torch.int32)
    init, fin, ck = perm[:n].clone(), perm[n:2 * n].clone(), perm[2 * n:2 * n + due].clone()
    init[-1], ck[1], ck[due // 2], ck[due - 1] = -1, -1, P, -7
    s[-1] = 0
    pool = torch.full((P, Hv, D, D), 7.0, device="cuda")
    pool[init[:-1].long()] = s[:-1]
    out, final, cks = kda.gdn_prefill(*d, s, _cu(lens), ckpt_stride=stride, ckpt_capacity=due, max_seq_len=hint)
    want = pool.clone()
    want[fin.long()] = final
    for j in range(due):
        if 0 <= ck[j] < P:
            want[ck[j].long()] = cks[j]
    o = kda.gdn_prefill_pooled(*d, pool, init.cuda(), fin.cuda(), _cu(lens), ckpt_stride=stride, ckpt_slots=ck.cuda(),
                               max_seq_len=hint)
    assert torch.equal(o, out) and torch.equal(pool, want)


def test_waits_give_up_in_segments_and_the_next_call_is_clean():
    """The passes and the join run on what a pass that gave up left; its status says so, the next call's does not."""
    lens = [1500, 700]
    x, s0, d, s = _inputs(lens, 1, 2, 128, 128, BF16, 97)
    desc = kda.make_gdn_desc(sum(lens), 1, 2, 128, 128, 2, kda.DTYPE_BF16, max_seq_len=1500)
    n = kda.gdn_workspace_size(desc)
    assert n > 4 * 2 * 2 * 128 * 128
    ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    kda.gdn_prefill(*d, s, _cu(lens), workspace=ws, wait_limit=1, max_seq_len=1500)
    assert kda.prefill_status(ws) == kda.STATUS_CODES["KDA_ERR_TIMEOUT"]
    out, final, _ = kda.gdn_prefill(*d, s, _cu(lens), workspace=ws, max_seq_len=1500)
    assert kda.prefill_status(ws) == 0
    want = ref.prefill(*x, s0.numpy(), lens)
    assert rel(f64(out), want[0]) <= tol_out(1500, BF16) and rel(f64(final), want[1]) <= tol_state(1500, BF16)
