"""The attention layers without a GPU: refusals before any launch, the scaled frequencies, and the plain forms that the
GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import attn_reference as ref
from linear_attention_serving_k1_gb300 import build, kda

INVALID, UNSUPPORTED, WORKSPACE = (kda.STATUS_CODES[x] for x in ("KDA_ERR_INVALID_ARG", "KDA_ERR_UNSUPPORTED", "KDA_ERR_WORKSPACE"))
P, O, WS = (ctypes.c_void_p(x) for x in (4096, 8192, 1 << 20))


@pytest.fixture(scope="module", params=["release", "debug"])
def lib(request):
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("no CUDA toolkit to build the library")
    build.build()
    return kda.load_library() if request.param == "release" else kda.load_debug_library()


# ---------------------------------------------------------------- refusals
def _desc(**kw):
    d = dict(T=256, Hq=8, Hkv=2, D=128, num_seqs=2, dtype_code=kda.DTYPE_BF16)
    d.update(kw)
    return kda.make_attn_desc(**d)


PAGED = dict(page_size=64, pages_per_seq=4, num_pages=9)
BAD_DESCS = [
    (dict(num_seqs=0), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(dtype_code=2), INVALID), (dict(max_seq_len=-1), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED), (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(PAGED, page_size=48), UNSUPPORTED), (dict(PAGED, page_size=8), UNSUPPORTED),
    (dict(PAGED, page_size=2048), UNSUPPORTED), (dict(PAGED, page_size=0), UNSUPPORTED), (dict(PAGED, pages_per_seq=0), INVALID),
    (dict(PAGED, num_pages=-1), INVALID), (dict(PAGED, pages_per_seq=1 << 28), UNSUPPORTED),
    (dict(PAGED, kv_dtype=kda.DTYPE_FP32), INVALID),
    (dict(PAGED, dtype_code=kda.DTYPE_FP32, kv_dtype=kda.DTYPE_E4M3), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_DESCS)
def test_bad_descs_are_refused(lib, kw, code):
    d = _desc(**kw)
    assert lib.kda_attn_workspace_size(ctypes.byref(d)) == 0 and lib.kda_attn_decode_workspace_size(ctypes.byref(d)) == 0
    tail = (ctypes.byref(d), WS, 1 << 30, None)
    assert lib.kda_attn_prefill(P, P, P, None, O, None, *tail) == code
    assert lib.kda_attn_prefill_paged(P, None, P, P, None, None, P, P, O, None, *tail) == code
    assert lib.kda_attn_decode(P, P, P, None, None, P, P, O, None, ctypes.byref(d), None, WS, 1 << 30, None) == code
    assert lib.kda_last_error()


def test_bad_calls_are_refused(lib):
    d, p = _desc(), _desc(**PAGED)
    n, m = (lib.kda_attn_workspace_size(ctypes.byref(x)) for x in (d, p))
    md = lib.kda_attn_decode_workspace_size(ctypes.byref(p))
    assert n >= 256 and n % 256 == 0 and m >= 256 and md % 256 == 0

    def prefill(q=P, k=P, v=P, cu=None, out=O, lse=None, desc=d, ws=WS, size=n):
        return lib.kda_attn_prefill(q, k, v, cu, out, lse, ctypes.byref(desc), ws, size, None)

    odd = ctypes.c_void_p(4100)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(out=P), dict(q=odd), dict(v=odd), dict(desc=p),
               dict(desc=_desc(T=255))):
        assert prefill(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(size=n - 1), dict(ws=ctypes.c_void_p((1 << 20) + 16))):
        assert prefill(**kw) == WORKSPACE, kw

    def paged(f, q=P, k=P, v=P, ks=None, vs=None, table=P, lens=P, out=O, desc=p, ws=WS, size=None):
        size = size if size is not None else m if f == "prefill" else md
        if f == "prefill":
            return lib.kda_attn_prefill_paged(q, None, k, v, ks, vs, table, lens, out, None, ctypes.byref(desc), ws, size, None)
        return lib.kda_attn_decode(q, k, v, ks, vs, table, lens, out, None, ctypes.byref(desc), None, ws, size, None)

    e = _desc(kv_dtype=kda.DTYPE_E4M3, **PAGED)
    for f in ("prefill", "decode"):
        for kw in (dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(out=P), dict(ks=P, vs=P),
                   dict(desc=e), dict(desc=e, ks=P), dict(k=odd), dict(desc=d), dict(desc=_desc(T=255, **PAGED))):
            assert paged(f, **kw) == INVALID, (f, kw)
        for kw in (dict(ws=None), dict(size=(m if f == "prefill" else md) - 1)):
            assert paged(f, **kw) == WORKSPACE, (f, kw)
    empty = _desc(T=0, **PAGED)
    # (no new token, but lengths to check: with a table they are read)
    for kw in (dict(lens=None), dict(table=None)):
        assert paged("prefill", desc=empty, **kw) == INVALID and paged("decode", desc=empty, **kw) == INVALID, kw
    assert lib.kda_attn_decode(None, P, P, None, None, P, P, None, None, ctypes.byref(empty), None, WS, 1 << 30, None) == 0


def test_bad_appends_are_refused(lib):
    def call(q=P, k=P, v=P, pos=P, ids=P, table=P, freq=P, qo=O, ko=None, kc=P, vc=P, ks=None, vs=None, **kw):
        f = dict(total_tokens=8, num_q_heads=4, num_kv_heads=2, head_dim=64, dtype=0, kv_dtype=0, rotary_dim=32, interleaved=0,
                 rope_scale=1.0, num_seqs=2, page_size=16, pages_per_seq=4, num_pages=8, q_stride=0, k_stride=0, v_stride=0)
        f.update(kw)
        return lib.kda_kv_append(q, k, v, pos, ids, table, freq, qo, ko, kc, vc, ks, vs, None, ctypes.byref(kda.AppendDesc(**f)), None)

    odd = ctypes.c_void_p(4100)
    e = dict(kv_dtype=kda.DTYPE_E4M3)
    for kw in (dict(total_tokens=-1), dict(num_q_heads=3), dict(rotary_dim=3), dict(rotary_dim=66), dict(rotary_dim=-2),
               dict(rotary_dim=0), dict(freq=None), dict(interleaved=2), dict(num_seqs=0), dict(pages_per_seq=0), dict(kv_dtype=1),
               dict(table=None), dict(kc=None), dict(vc=None), dict(ids=None), dict(v=None), dict(ks=P, vs=P), e, dict(e, ks=P),
               dict(k=None), dict(pos=None), dict(q=None), dict(qo=None), dict(q_stride=8), dict(q_stride=260), dict(k=odd),
               dict(qo=odd), dict(kc=odd), dict(qo=P, q_stride=512), dict(ko=P, k_stride=512), dict(ko=O, qo=O),
               dict(table=None, kc=None, vc=None, ks=P, vs=P)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(head_dim=96, rotary_dim=32), dict(page_size=24), dict(page_size=8), dict(e, dtype=1, ks=P, vs=P),
               dict(total_tokens=1 << 31)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(total_tokens=0) == 0


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_scales_that_are_not_aligned_are_refused(lib, which):
    """Decode copies them 16 bytes at a time; the other calls over such a cache refuse it too."""
    at = {x: ctypes.c_void_p(4100) if x == which else P for x in ("k_scale", "v_scale")}
    scales = (at["k_scale"], at["v_scale"])
    d = _desc(kv_dtype=kda.DTYPE_E4M3, **PAGED)
    tail = (P, P, O, None, ctypes.byref(d))
    assert lib.kda_attn_decode(P, P, P, *scales, *tail, None, WS, 1 << 30, None) == INVALID
    assert b"aligned" in lib.kda_last_error()
    assert lib.kda_attn_prefill_paged(P, None, P, P, *scales, *tail, WS, 1 << 30, None) == INVALID
    assert b"aligned" in lib.kda_last_error()
    a = kda.AppendDesc(8, 4, 2, 64, kda.DTYPE_BF16, kda.DTYPE_E4M3, 0, 0, 1.0, 2, 16, 4, 8, 0, 0, 0)
    assert lib.kda_kv_append(P, P, P, P, P, P, None, O, None, P, P, *scales, None, ctypes.byref(a), None) == INVALID
    assert b"aligned" in lib.kda_last_error()


@pytest.mark.parametrize("scales", [(P, None), (None, P), (P, P)])
@pytest.mark.parametrize("pages", [0, 9])
def test_scales_without_an_e4m3_cache_are_refused(lib, scales, pages):
    """Also one alone, and without a page."""
    for code in (kda.DTYPE_BF16, kda.DTYPE_FP32):
        d = _desc(dtype_code=code, **dict(PAGED, num_pages=pages))
        tail = (P, P, O, None, ctypes.byref(d))
        assert lib.kda_attn_decode(P, P, P, *scales, *tail, None, WS, 1 << 30, None) == INVALID
        assert b"no other" in lib.kda_last_error()
        assert lib.kda_attn_prefill_paged(P, None, P, P, *scales, *tail, WS, 1 << 30, None) == INVALID
        assert b"no other" in lib.kda_last_error()


def test_binding_refuses_cpu_tensors_and_shapes():
    q, k = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.attn_prefill(q, k, k)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kv_append(q, k, k, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="bf16 or fp32"):
        kda.attn_prefill(q.half(), k.half(), k.half())
    cache = torch.zeros(3, 2, 16, 128, dtype=torch.float32)
    with pytest.raises(ValueError):
        kda.attn_decode(q, cache, cache, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("name", ["page_table", "v_cache", "k_scale", "v_scale"])
def test_binding_refuses_parts_of_a_cache(name):
    """A part of a cache without its keys would have been left as it was, in silence."""
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="go with k_cache"):
        kda.kv_append(None, k, k, pos, seq_ids=pos, **{name: torch.zeros(1, 2, 16, 128)})


@pytest.mark.parametrize("scale", [0.0, -1.0, math.inf, math.nan])
def test_binding_refuses_scales(scale):
    """0 is the C call's word for the default, and no scale of a caller's."""
    with pytest.raises(ValueError, match="scale"):
        kda._scale_arg(scale)
    assert kda._scale_arg(None) == 0.0 and kda._scale_arg(0.25) == 0.25


@pytest.mark.parametrize("scale", [1e-50, 1e39, -1e-50])
def test_binding_refuses_scales_that_fp32_does_not_hold(scale):
    """The first would have become 0, the default."""
    with pytest.raises(ValueError, match="scale"):
        kda._scale_arg(scale)
    assert kda._scale_arg(1e-40) == 1e-40


# ---------------------------------------------------------------- frequencies
def test_rope_frequencies():
    f, s = kda.rope_frequencies(128, 10000.0)
    want = torch.tensor([10000.0 ** (-2 * i / 128) for i in range(64)], dtype=torch.float64)
    assert s == 1.0 and f.dtype == torch.float32 and (f.double() / want - 1).abs().max() <= ref.EPS32
    lin, _ = kda.rope_frequencies(128, scaling="linear", factor=4.0)
    assert torch.equal(lin, (want / 4).float())
    b, _ = kda.rope_frequencies(64, 500000.0, scaling="base", factor=8.0)
    plain, _ = kda.rope_frequencies(64, 500000.0)
    assert b[0] == 1.0 and abs(float(plain[-1] / b[-1]) - 8) < 1e-5
    p, s = kda.rope_frequencies(128, 10000.0, scaling="parts", factor=16.0, original_len=4096)
    assert abs(s - (0.1 * math.log(16) + 1)) < 1e-12
    turns = 4096 * want / (2 * math.pi)
    assert torch.equal(p[turns > 32], want[turns > 32].float())
    assert (p[turns < 1].double() * 16 / want[turns < 1] - 1).abs().max() < 1e-6
    assert (p.double() <= want * (1 + 1e-6)).all() and (p.double() * 16 >= want * (1 - 1e-6)).all()
    for kw in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, scaling="parts"),
               dict(rotary_dim=8, scaling="other"), dict(rotary_dim=2, scaling="base"), dict(rotary_dim=8, base=1.0)):
        with pytest.raises(ValueError):
            kda.rope_frequencies(**kw)


# ---------------------------------------------------------------- the plain forms themselves
def test_reference_rotation_keeps_lengths_and_relative_positions():
    g = torch.Generator().manual_seed(1)
    x, y = torch.randn(2, 1, 3, 32, generator=g, dtype=torch.float64)
    f, _ = kda.rope_frequencies(20)
    for inter in (False, True):
        at = lambda z, p: ref.rotate(z, torch.tensor([p]), f, inter, 1.0)  # noqa: E731
        assert (at(x, 12345).norm(dim=-1) - x.norm(dim=-1)).abs().max() < 1e-12
        assert ((at(x, 105) * at(y, 98)).sum(-1) - (at(x, 7) * at(y, 0)).sum(-1)).abs().max() < 1e-9
        assert torch.equal(at(x, 0), x) and torch.equal(at(x, 9)[..., 20:], x[..., 20:])


def test_reference_rows_of_eight_bits():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(500, 64, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-40, 40, (500, 1), generator=g))
    s = ref.scale_of(x)
    top = x.abs().amax(-1)
    assert (top <= 448 * s).all() and (top > 224 * s).all()
    c = ref.codes(x, s)
    assert torch.equal(c.float(), (x / s[:, None]).float().to(ref.F8).float())
    edge = torch.tensor([[448.0], [449.0], [0.0], [2.0 ** -130], [math.inf], [math.nan]], dtype=torch.float64)
    assert ref.scale_of(edge)[:4].tolist() == [1.0, 2.0, 2.0 ** -126, 2.0 ** -126] and ref.scale_of(edge)[4:].isnan().all()


def test_reference_attention_closed_forms():
    k, v = torch.zeros(5, 1, 4, dtype=torch.float64), torch.arange(20, dtype=torch.float64).reshape(5, 1, 4)
    q = torch.ones(5, 2, 4, dtype=torch.float64)
    out, lse, _, _ = ref.attend(q, k, v, 0, 0.5)     # equal scores: running means
    assert torch.allclose(out[:, 1], torch.cumsum(v[:, 0], 0) / torch.arange(1, 6)[:, None])
    assert torch.allclose(lse[:, 0], torch.log(torch.arange(1, 6, dtype=torch.float64)))
    out, lse, _, _ = ref.attend(q, k, v, -2, 0.5)    # rows before the first key
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all() and torch.equal(out[2, 0], v[0, 0])
