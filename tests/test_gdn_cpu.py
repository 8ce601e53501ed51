"""The grouped gated delta rule and the batch plan without a GPU: refused calls
(on the host, before anything is launched) and the workspace size."""
import ctypes

import pytest
import torch

from linear_attention_serving_k1_gb300 import build, kda

P = ctypes.c_void_p(4096)
O = ctypes.c_void_p(1 << 16)
WS = ctypes.c_void_p(1 << 20)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5


@pytest.fixture(scope="module")
def lib():
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("no CUDA toolkit to build the library")
    build.build()
    return kda.load_library()


def _desc(**kw):
    d = dict(T=256, Hk=2, Hv=4, Dk=128, Dv=128, num_seqs=1, dtype_code=kda.DTYPE_BF16)
    d.update(kw)
    return kda.make_gdn_desc(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(Hk=0), INVALID),
    (dict(Hk=3), INVALID), (dict(Hv=0), INVALID), (dict(Dk=96), UNSUPPORTED), (dict(Dk=256), UNSUPPORTED),
    (dict(Dv=96), UNSUPPORTED), (dict(Dv=0), UNSUPPORTED), (dict(Dv=576), UNSUPPORTED), (dict(dtype_code=3), INVALID),
    (dict(ckpt_stride=100), INVALID), (dict(ckpt_stride=-64), INVALID), (dict(ckpt_capacity=-1), INVALID),
    (dict(max_seq_len=-1), INVALID), (dict(num_seqs=1 << 30), UNSUPPORTED)])
def test_invalid_desc(lib, kw, code):
    d = _desc(**kw)
    assert lib.kda_gdn_workspace_size(ctypes.byref(d)) == 0
    assert lib.kda_gdn_prefill(P, P, P, P, P, None, None, O, None, None, ctypes.byref(d), WS, 1 << 30, None) == code
    assert lib.kda_last_error()


def test_workspace_is_small(lib):
    assert 0 < lib.kda_gdn_workspace_size(ctypes.byref(_desc(T=1 << 20, num_seqs=1000))) < 64 * 1000


def test_prefill_rejects_before_launch(lib):
    def call(d=None, q=P, out=O, init=None, ckpts=None, ws=WS, ws_bytes=1 << 20):
        return lib.kda_gdn_prefill(q, P, P, P, P, init, None, out, None, ckpts, ctypes.byref(d or _desc()), ws,
                                   ws_bytes, None)
    assert call(q=None) == INVALID
    assert call(out=P) == INVALID                                     # out aliases q
    assert call(q=ctypes.c_void_p(4100)) == INVALID                   # alignment
    assert call(out=ctypes.c_void_p(65540)) == INVALID
    assert call(init=ctypes.c_void_p(4100)) == INVALID
    assert call(ws=None) == WORKSPACE
    assert call(ws=ctypes.c_void_p((1 << 20) + 8)) == WORKSPACE
    assert call(ws_bytes=256) == WORKSPACE
    assert call(_desc(T=255, num_seqs=2)) == INVALID                  # does not divide
    assert call(_desc(ckpt_stride=64, ckpt_capacity=1)) == INVALID    # no ckpts
    assert lib.kda_gdn_prefill(P, P, P, P, P, None, None, O, None, None, None, WS, 1 << 20, None) == INVALID


def test_pooled_rejects_before_launch(lib):
    def call(d=None, pool=P, slots=8, init=None, ckpt=None):
        return lib.kda_gdn_prefill_pooled(P, P, P, P, P, None, O, pool, ctypes.c_int64(slots), init, None, ckpt,
                                          ctypes.byref(d or _desc()), WS, 1 << 20, None)
    assert call(slots=-1) == INVALID
    assert call(pool=None, init=P) == INVALID
    assert call(pool=ctypes.c_void_p(4104)) == INVALID
    assert call(_desc(ckpt_stride=64, ckpt_capacity=1)) == INVALID


def test_decode_rejects_before_launch(lib):
    def call(q=P, state=P, slots=None, pool=0, out=O, N=2, Hk=2, Hv=4, Dk=128, Dv=128, dtype=0, m=None):
        if m is None:
            return lib.kda_gdn_decode(q, P, P, P, P, state, ctypes.c_int64(pool), slots, out, N, Hk, Hv, Dk, Dv, dtype,
                                      None, None)
        return lib.kda_gdn_decode_multi(q, P, P, P, P, state, ctypes.c_int64(pool), slots, None, out, N, m, Hk, Hv, Dk,
                                        Dv, dtype, None, None)
    for m in (None, 3):
        assert call(m=m, N=-1) == INVALID
        assert call(m=m, Hk=3) == INVALID
        assert call(m=m, Dk=96) == UNSUPPORTED
        assert call(m=m, Dv=100) == UNSUPPORTED
        assert call(m=m, dtype=4) == INVALID
        assert call(m=m, q=None) == INVALID
        assert call(m=m, state=ctypes.c_void_p(4104)) == INVALID
        assert call(m=m, out=P) == INVALID
        assert call(m=m, slots=P, pool=-1) == INVALID
        assert call(m=m, N=1 << 30) == UNSUPPORTED
        assert call(m=m, N=0) == 0
    assert call(m=-1) == INVALID
    assert call(m=0) == 0


def test_plan_rejects_before_launch(lib):
    def call(lens=P, slots=P, free=P, num_free=4, head=P, N=4, T=64, stride=64, cap=4, table=None, cols=0, cu=O,
             init=O, ckpt=O, ids=O, head_out=O, slots_out=P):
        return lib.kda_plan_batch(lens, None, None, slots, free, num_free, head, N, T, stride, cap, table, cols, cu,
                                  init, slots_out, O, ckpt, ids, O, head_out, None, None)
    for kw, code in ((dict(N=0), INVALID), (dict(N=16385), UNSUPPORTED), (dict(T=-1), INVALID),
                     (dict(T=1 << 31), UNSUPPORTED), (dict(stride=-64), INVALID), (dict(stride=96), INVALID),
                     (dict(cap=-1), INVALID), (dict(cap=1 << 31), INVALID), (dict(num_free=-1), INVALID),
                     (dict(lens=None), INVALID), (dict(slots=None), INVALID), (dict(head=None), INVALID),
                     (dict(head_out=None), INVALID), (dict(cu=None), INVALID), (dict(free=None), INVALID),
                     (dict(ckpt=None), INVALID), (dict(ids=None), INVALID), (dict(cols=-1), INVALID),
                     (dict(table=O, cols=0), INVALID), (dict(cu=P), INVALID), (dict(init=P), INVALID),
                     (dict(slots_out=O), INVALID)):
        assert call(**kw) == code, kw


def test_python_binding_checks_shapes(lib):
    """Wrong shapes, types and devices are refused by the binding before the library is called."""
    T, Hk, Hv, Dk, Dv = 8, 2, 4, 64, 64
    q, k, v = torch.zeros(T, Hk, Dk), torch.zeros(T, Hk, Dk), torch.zeros(T, Hv, Dv)
    g, beta, S = torch.zeros(T, Hv), torch.zeros(T, Hv), torch.zeros(T, Hv, Dk, Dv)
    ok = dict(q=q, k=k, v=v, g=g, beta=beta)
    for name, bad in (("k", k.bfloat16()), ("k", k[:4]), ("v", v[:4]), ("g", g[:, :2]), ("g", g.double()),
                      ("beta", beta[:, :1]), ("q", q.half()), ("q", q[0])):
        with pytest.raises(ValueError):
            kda.gdn_decode(**dict(ok, **{name: bad}), state=S)
        with pytest.raises(ValueError):
            kda.gdn_prefill(**dict(ok, **{name: bad}))
    with pytest.raises(ValueError):
        kda.gdn_decode(**ok, state=S[:4])
    with pytest.raises(ValueError):
        kda.gdn_decode(**ok, state=S, slot_ids=torch.zeros(T, dtype=torch.int64))
    with pytest.raises(ValueError):
        kda.gdn_prefill(**ok, init_state=S)
    with pytest.raises(ValueError):
        kda.gdn_prefill(**ok, cu_seqlens=torch.zeros(2))
    with pytest.raises(ValueError):
        kda.gdn_prefill(**ok, ckpt_stride=64, ckpts=torch.zeros(1, Hv, Dk, Dv), ckpt_capacity=2)
    with pytest.raises(ValueError):
        kda.gdn_prefill_pooled(**ok, state_pool=S, init_slots=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):   # tensors that are not on a GPU
        kda.gdn_decode(**ok, state=S)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.plan_batch(i, i[:3], total_tokens=4)
    with pytest.raises(ValueError):
        kda.plan_batch(i, i.clone(), total_tokens=4, past=i.long())
    with pytest.raises(ValueError):
        kda.plan_batch(i, i.clone(), total_tokens=4)   # not on a GPU


def test_workspace_and_stream_of_another_device_are_refused(lib):
    """Before the library is called (stand-ins for a tensor and a stream of a second GPU)."""
    class Other:
        device = torch.device("cuda", 1)
        is_cuda, cuda_stream = True, 0

        def __getattr__(self, name):
            raise AssertionError(f"{name} was used")

    d = _desc()
    with pytest.raises(ValueError, match="workspace"):
        kda._gdn_workspace(d, Other(), torch.device("cuda", 0), None)
    with pytest.raises(ValueError, match="stream"):
        kda._call("kda_gdn_decode", 0, Other())
