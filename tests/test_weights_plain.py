"""CPU checks of the calls that accumulate attention weights and of the eviction: their argument
checks (C ABI and Python), and the tests' plain forms against the oracle and by hand."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
import plain_weights as pw
from cases import bf16_to_f64
from test_abi import BAD, P, _shape
from test_oracle_multi import Multi


@pytest.fixture(scope="module")
def lib():
    from paged_decode_attention_kv_gb300 import build
    build.build()
    return da.load_library()


def call(lib, name, **kw):
    a = dict(q=P, k_new=P, v_new=P, kc=P, vc=P, w=P, bt=P, sl=P, ql=None, sinks=P, window=0, scale=0.125, out=P,
             s=_shape(), T=4, page=16, maxp=16, npages=64, maxlen=200)
    a.update(kw)
    tail = [a["page"], a["maxp"], a["npages"], a["maxlen"], None]
    head = [a["q"], a["k_new"], a["v_new"], a["kc"]]
    if name == "fp8":
        return lib.decode_attn_paged_fp8_weights(*head, a["w"], a["bt"], a["sl"], a["sinks"], a["window"], a["scale"],
                                                 a["out"], a["s"], *tail)
    if name == "multi":
        return lib.decode_attn_paged_multi_weights(*head, a["vc"], a["w"], a["bt"], a["sl"], a["ql"], a["sinks"],
                                                   a["window"], a["scale"], a["out"], a["s"], a["T"], *tail)
    return lib.decode_attn_paged_weights(*head, a["vc"], a["w"], a["bt"], a["sl"], a["sinks"], a["window"], a["scale"],
                                         a["out"], a["s"], *tail)


@pytest.mark.parametrize("name", ["bf16", "fp8", "multi"])
def test_weights_argument_validation(lib, name):
    assert call(lib, name, w=None) == -1
    assert call(lib, name, w=BAD) == -1
    assert call(lib, name, q=None) == -1
    assert call(lib, name, q=BAD) == -1
    assert call(lib, name, k_new=None) == -1
    assert call(lib, name, kc=None) == -1
    assert call(lib, name, bt=None) == -1
    assert call(lib, name, sl=None) == -1
    assert call(lib, name, out=None) == -1
    for bad in (0.0, -0.125, float("nan"), float("inf")):
        assert call(lib, name, scale=bad) == -1
    assert call(lib, name, window=-1) == -1
    assert call(lib, name, page=32) == -2
    assert call(lib, name, maxlen=16 * 16 + 1) == -1
    assert call(lib, name, npages=0) == -1
    assert call(lib, name, s=_shape(D=128)) == -2
    assert call(lib, name, s=_shape(Hq=24, Hkv=1)) == -2
    assert call(lib, name, s=_shape(Hq=6, Hkv=4)) == -1
    assert call(lib, name, s=_shape(B=2048)) == -2
    assert call(lib, name, s=_shape(B=0)) == 0
    if name == "multi":
        assert call(lib, name, T=0) == -1
        assert call(lib, name, T=-3) == -1
        assert call(lib, name, T=5000) == -2


def evict(lib, fp8=False, **kw):
    a = dict(kc=P, vc=P, w=P, bt=P, sl=P, nl=ctypes.c_void_p(0x20000), kept=P, keep=32, first=4, last=8,
             s=_shape(Hq=1, Hkv=1), page=16, maxp=16, npages=64, maxlen=200)
    a.update(kw)
    args = [a["w"], a["bt"], a["sl"], a["nl"], a["kept"], a["keep"], a["first"], a["last"], a["s"], a["page"], a["maxp"],
            a["npages"], a["maxlen"], None]
    return lib.kv_evict_fp8(a["kc"], *args) if fp8 else lib.kv_evict(a["kc"], a["vc"], *args)


@pytest.mark.parametrize("fp8", [False, True])
def test_evict_argument_validation(lib, fp8):
    for name in ("kc", "w", "bt", "sl", "nl", "kept"):
        assert evict(lib, fp8, **{name: None}) == -1
    if not fp8:
        assert evict(lib, vc=None) == -1
        assert evict(lib, vc=BAD) == -1
    assert evict(lib, fp8, kc=BAD) == -1
    assert evict(lib, fp8, w=BAD) == -1
    assert evict(lib, fp8, keep=0) == -1
    assert evict(lib, fp8, first=-1) == -1
    assert evict(lib, fp8, last=-1) == -1
    assert evict(lib, fp8, first=20, last=13) == -1              # more than keep
    assert evict(lib, fp8, first=33, last=0) == -1
    assert evict(lib, fp8, first=2 ** 31 - 1, last=2 ** 31 - 1) == -1
    assert evict(lib, fp8, nl=P) == -1                           # new_lens is seq_lens
    assert evict(lib, fp8, nl=ctypes.c_void_p(0x10004)) == -1    # overlapping
    assert evict(lib, fp8, page=8) == -2
    assert evict(lib, fp8, maxlen=16 * 16 + 1) == -1
    assert evict(lib, fp8, maxp=0) == -1
    assert evict(lib, fp8, s=_shape(Hq=1, Hkv=1, D=32)) == -2
    assert evict(lib, fp8, s=_shape(Hq=1, Hkv=1, B=0)) == 0


def test_workspace_bytes(lib):
    assert da.decode_attn_weights_workspace_bytes(2, 8, 1) >= 2 * 8 * 4
    assert da.decode_attn_weights_workspace_bytes(2, 8, 1, 4096) >= 2 * 8 * 4096 * 4
    assert da.decode_attn_weights_workspace_bytes(2, 8, 3) == 0
    assert da.decode_attn_weights_workspace_bytes(2, 8, 1, 4097) == 0
    assert da.kv_evict_workspace_bytes(2, 8, 1024) >= 2 * 8 * 1024 * 8
    assert da.kv_evict_workspace_bytes(2, 8, 0) == 0


def test_python_checks_name_the_tensor(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, kn = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 1, 64, dtype=bf)
    pool, w = torch.zeros(4, 1, 16, 64, dtype=bf), torch.zeros(4, 1, 16, dtype=f32)
    bt, sl = torch.zeros(2, 2, dtype=i32), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="k_cache"):     # not on a GPU
        da.decode_attn_paged_weights(q, kn, kn, pool, pool, w, bt, sl, None, 0, 0.125, q)
    with pytest.raises(ValueError, match="cache"):
        da.decode_attn_paged_weights(q, kn, kn, pool[0], pool, w, bt, sl, None, 0, 0.125, q)
    with pytest.raises(ValueError, match="kv_cache"):
        da.kv_evict_fp8(torch.zeros(4, 1, 100, dtype=torch.uint8), w, bt, sl, sl, bt)


# ---------------------------------------------------------------- the plain forms
@pytest.mark.parametrize("window", [0, 3, 20])
def test_plain_step_gives_the_oracles_output(window):
    m = Multi(910 + window, 8, 2, [5, 17, 33, 0], [3, 1, 4, 0], 4)
    ref = m.run(window)
    for b, L in enumerate(m.lens):
        if L == 0:
            continue
        out, mass, seen = pw.step(bf16_to_f64(m.q[b]), bf16_to_f64(m.c.hist_k[b, :L]), bf16_to_f64(m.c.hist_v[b, :L]), int(L),
                                  int(m.n[b]), m.sinks.astype(np.float64), window, m.c.scale)
        np.testing.assert_allclose(out, ref[b], rtol=0, atol=1e-12)
        # every row's probabilities and its sink's share make one
        assert np.all(mass.sum(0) < m.n[b] * 4) and np.all(mass[~seen] == 0) and np.all(mass[seen] > 0)
        _, no_sink, _ = pw.step(bf16_to_f64(m.q[b]), bf16_to_f64(m.c.hist_k[b, :L]), bf16_to_f64(m.c.hist_v[b, :L]), int(L),
                                int(m.n[b]), None, window, m.c.scale)
        np.testing.assert_allclose(no_sink.sum(0), m.n[b] * 4, rtol=1e-12)


def test_plain_eviction_by_hand():
    w = np.array([9, 1, 5, 2, 5, 7, 0, 5, 3, 8], np.float32)
    # first 1, last 2 stay; of cells 1..7 (1 5 2 5 7 0 5) the largest three: 5, then 2 and 4 (ties, lowest)
    assert pw.kept_cells(w, 10, 6, 1, 2).tolist() == [0, 4, 2, 5, 8, 9]
    assert pw.kept_cells(w, 4, 6, 1, 2).tolist() == [0, 1, 2, 3, -1, -1]
    assert pw.kept_cells(w, 10, 3, 1, 2).tolist() == [0, 8, 9]
    w[2] = np.nan
    assert pw.kept_cells(w, 10, 2, 0, 0).tolist() == [0, 9]
    w[:] = 0
    w[3] = -0.0
    assert pw.kept_cells(w, 10, 5, 0, 0).tolist() == [0, 1, 2, 3, 4]
