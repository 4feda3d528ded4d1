"""CPU: what qk_norm_rope, kv_append_fp8, kv_read_fp8 and decode_attn_paged_fp8_multi refuse, at the C ABI (before
the first CUDA call) and in the Python binding."""
import ctypes

import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from test_abi import BAD, P, _shape


@pytest.fixture(scope="module")
def lib():
    from paged_decode_attention_kv_gb300 import build
    build.build()
    return da.load_library()


def rotate(lib, q={}, k={}, v=None, **kw):
    def rows(change, heads):
        a = dict(in_=0x10000, out=0x20000, in_stride=heads * 64, out_stride=heads * 64)
        a.update(change)
        return ctypes.byref(da.da_rows(a["in_"], a["out"], a["in_stride"], a["out_stride"]))
    a = dict(n=4, Hq=8, Hkv=2, D=64, pos=P, axes=1, table=None, cos=P, sin=P, most=100, qw=P, kw=P, eps=1e-6)
    a.update(kw)
    return lib.qk_norm_rope(None if q is None else rows(q, 8), None if k is None else rows(k, 2), None if v is None else rows(v, 2), a["n"], a["Hq"],
                            a["Hkv"], a["D"], a["pos"], a["axes"], a["table"], a["cos"], a["sin"], a["most"], a["qw"], a["kw"], a["eps"], None)


def test_rotate_refusals(lib):
    for change in (dict(q=None), dict(k=None), dict(q=dict(in_=None)), dict(q=dict(out=0x10008)), dict(k=dict(in_=0x10002)),
                   dict(q=dict(in_stride=511)), dict(q=dict(in_stride=448)), dict(k=dict(out_stride=64)), dict(v=dict(out_stride=64)),
                   dict(v=dict(in_=None)), dict(n=-1), dict(Hq=0), dict(Hkv=-1), dict(pos=None), dict(cos=None), dict(sin=BAD),
                   dict(most=0), dict(qw=BAD), dict(kw=BAD), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                   dict(axes=0), dict(axes=4, table=bytes(32)), dict(axes=2), dict(axes=2, table=bytes([0] * 31 + [2]))):
        assert rotate(lib, **change) == -1, change
    assert rotate(lib, D=128) == -2
    assert rotate(lib, Hq=1025, q=dict(in_stride=65600, out_stride=65600)) == -2
    assert rotate(lib, n=0) == 0
    assert rotate(lib, n=0, pos=None, q=dict(in_=None, out=None), k=dict(in_=None, out=None)) == 0  # empty tensors have no address
    assert rotate(lib, n=0, axes=3, table=bytes([0, 1, 2, 2] * 8)) == 0


def append(lib, **kw):
    a = dict(k=P, v=P, kv=P, bt=P, sl=P, ql=None, window=0, rule=1, s=_shape(), T=4, page=16, maxp=16, npages=64, maxlen=200)
    a.update(kw)
    return lib.kv_append_fp8(a["k"], a["v"], a["kv"], a["bt"], a["sl"], a["ql"], a["window"], a["rule"], a["s"], a["T"], a["page"], a["maxp"],
                             a["npages"], a["maxlen"], None)


def read(lib, **kw):
    a = dict(kv=P, bt=P, sl=P, st=None, window=0, k=P, v=P, rows=40, s=_shape(), page=16, maxp=16, npages=64, maxlen=200)
    a.update(kw)
    return lib.kv_read_fp8(a["kv"], a["bt"], a["sl"], a["st"], a["window"], a["k"], a["v"], a["rows"], a["s"], a["page"], a["maxp"], a["npages"],
                           a["maxlen"], None)


def multi(lib, **kw):
    a = dict(q=P, k=P, v=P, kv=P, bt=P, sl=P, ql=None, sinks=P, window=0, scale=0.125, rule=1, out=P, s=_shape(), T=4, page=16, maxp=16,
             npages=64, maxlen=200)
    a.update(kw)
    return lib.decode_attn_paged_fp8_multi(a["q"], a["k"], a["v"], a["kv"], a["bt"], a["sl"], a["ql"], a["sinks"], a["window"], a["scale"], a["rule"],
                                           a["out"], a["s"], a["T"], a["page"], a["maxp"], a["npages"], a["maxlen"], None)


def test_refusals_of_the_cache_calls(lib):
    for call in (append, read, multi):
        for change in (dict(kv=None), dict(kv=BAD), dict(sl=None), dict(k=None), dict(v=BAD), dict(maxp=0), dict(npages=0), dict(maxlen=16 * 16 + 1),
                       dict(maxlen=-1), dict(s=_shape(B=-1))):
            assert call(lib, **change) == -1, (call.__name__, change)
        for change in (dict(page=32), dict(s=_shape(D=128)), dict(s=_shape(B=2048)), dict(npages=2 ** 31 - 1, s=_shape(Hq=8, Hkv=8))):
            assert call(lib, **change) == -2, (call.__name__, change)
        assert call(lib, s=_shape(B=0)) == 0
    for call in (append, read):
        assert call(lib, bt=None) == -1                        # a ring of no cells
        assert call(lib, bt=None, window=24) == -2             # not whole blocks
        assert call(lib, bt=None, window=32, s=_shape(B=0)) == 0
    for call in (append, multi):
        assert call(lib, T=0) == -1
        assert call(lib, rule=2) == -1
    assert read(lib, rows=-1) == -1
    assert read(lib, rows=0) == 0
    assert read(lib, rows=0, k=None, v=None) == 0                  # empty tensors have no address
    for change in (dict(q=None), dict(out=BAD), dict(bt=None), dict(scale=0.0), dict(scale=-0.125), dict(scale=float("inf")), dict(scale=float("nan")),
                   dict(window=-1), dict(s=_shape(Hq=6, Hkv=4))):
        assert multi(lib, **change) == -1, change
    assert multi(lib, T=4097) == -2
    assert multi(lib, s=_shape(Hq=24, Hkv=1)) == -2


def test_the_binding_names_what_it_refuses(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    kv = torch.zeros(3, 4, 2176, dtype=torch.uint8)
    cos = torch.zeros(8, 32)
    with pytest.raises(ValueError, match="q must be"):
        da.qk_norm_rope(x, x, i, cos, cos, x, x)               # not on a GPU
    with pytest.raises(ValueError, match="given together"):
        da.qk_norm_rope(x, x, i, cos, cos, x, x, v=x)
    with pytest.raises(ValueError, match=r"q and k are"):
        da.qk_norm_rope(x[0], x[0], i, cos, cos, x, x)
    with pytest.raises(ValueError, match="seq_lens must be"):
        da.kv_append_fp8(x, x, kv, i, i.view(1, 2))
    with pytest.raises(ValueError, match="kv_cache is"):
        da.kv_read_fp8(kv, i, x, x)
    with pytest.raises(ValueError, match="q is"):
        da.decode_attn_paged_fp8_multi(x, x, x, kv, i.view(1, 2), i, None, 0, 0.125, x)
    for bad in ((16, 8), (16, 8, 9), (40, -8, 0)):
        with pytest.raises(ValueError, match="sections"):
            da._pair_axes(3, bad, False)
    assert da._pair_axes(3, (8, 12, 12), True)[:4] == bytes([0, 1, 2, 0])
    assert da._pair_axes(3, (8, 12, 12), False) == bytes([0] * 8 + [1] * 12 + [2] * 12)
