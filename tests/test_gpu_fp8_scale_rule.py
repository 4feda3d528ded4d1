"""GPU: decode_attn_paged_fp8_weights with DA_FP8_SCALE_DIVIDE is decode_attn_paged_fp8 bit for bit, the
appended token's bytes and the output alike; a cache that both calls append to in turn is the one
that decode_attn_paged_fp8 alone leaves."""
import numpy as np
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from cases import paged_identity, shuffle_pages
from paged_decode_attention_kv_gb300 import workloads as wl
from test_gpu_decode import DEV, dev, dev_bits
from test_gpu_weights import EDGE, one_token

pytestmark = pytest.mark.gpu


def both(m, window=0, sinks=True, seed=1):
    """The call with weights and the one without on copies of one random cache of finite codes."""
    c = m.c
    kp, vp, bt = shuffle_pages(*paged_identity(c, c.lens), seed, spare=2)
    rng = np.random.default_rng(seed)
    kv = rng.integers(0, 256, (kp.shape[0], c.Hkv, 2176), dtype=np.uint8)
    kv[..., :2048][(kv[..., :2048] & 127) == 127] -= 1
    kv[..., 2048:] = ((2 + rng.random(kv.shape[:2] + (32,))) / 448).astype(np.float32).view(np.uint8)
    a, b = dev(kv), dev(kv)
    q, kn, vn, btd, sl = dev_bits(m.q)[:, 0].contiguous(), dev_bits(c.k_new), dev_bits(c.v_new), dev(bt), dev(c.lens)
    sk, out, ref = dev(c.sinks) if sinks else None, torch.empty_like(q), torch.empty_like(q)
    w = torch.zeros((kp.shape[0], c.Hkv, 16), device=DEV)
    da.decode_attn_paged_fp8_weights(q, kn, vn, a, w, btd, sl, sk, window, c.scale, out, scale_rule=da.DA_FP8_SCALE_DIVIDE)
    da.decode_attn_paged_fp8(q, kn, vn, b, btd, sl, sk, window, c.scale, ref)
    assert da.decode_attn_device_status() == 0
    assert torch.equal(a, b)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    return kv, a


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (8, 8), (16, 1), (32, 4), (4, 2)])
@pytest.mark.parametrize("window", [0, 7, 100])
def test_divide_is_the_call_without_weights(Hq, Hkv, window):
    both(one_token(4000 + Hq + window, Hq, Hkv, EDGE), window, sinks=window != 7, seed=Hq)


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 1)])
def test_divide_over_every_mantissa(Hq, Hkv):
    """Rows whose largest value takes every bf16 mantissa: for 71 of the 128 the two rules differ."""
    m = one_token(4020 + Hq, Hq, Hkv, [1 + i for i in range(128)])
    gen = np.random.default_rng(Hq)
    for b in range(128):
        for x in (m.c.k_new, m.c.v_new):
            x[b] = (gen.integers(0, 128, x[b].shape) | 0x3f00 | gen.integers(0, 2, x[b].shape) << 15).astype(np.uint16)
            x[b, :, 5] = 0x4000 | b
    both(m)


def test_divide_on_two_ctas_per_sm():
    both(one_token(4030, 64, 8, [33000, 3001]))


def test_weights_on_every_other_step():
    """40 steps of three sequences, with weights on every other one."""
    gen = wl.cpu_generator(4040)
    B, Hq, Hkv, pages = 3, 16, 2, 24
    bt = dev(np.arange(B * 4, dtype=np.int32).reshape(B, 4))
    a, b = (torch.zeros((pages, Hkv, 2176), dtype=torch.uint8, device=DEV) for _ in range(2))
    w, lens = torch.zeros((pages, Hkv, 16), device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    for step in range(40):
        q, kn, vn = (dev(wl.randn_bf16((B, h, 64), gen)) for h in (Hq, Hkv, Hkv))
        lens += 1
        out, ref = torch.empty_like(q), torch.empty_like(q)
        if step % 2:
            da.decode_attn_paged_fp8_weights(q, kn, vn, a, w, bt, lens, None, 0, 0.125, out, scale_rule=da.DA_FP8_SCALE_DIVIDE)
        else:
            da.decode_attn_paged_fp8(q, kn, vn, a, bt, lens, None, 0, 0.125, out)
        da.decode_attn_paged_fp8(q, kn, vn, b, bt, lens, None, 0, 0.125, ref)
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    assert torch.equal(a, b)
    assert da.decode_attn_device_status() == 0


def test_other_rules_are_refused():
    m = one_token(4050, 16, 2, [40, 7])
    with pytest.raises(da.DecodeAttnError) as e:
        q, sl = dev_bits(m.q)[:, 0].contiguous(), dev(m.lens)
        kv, w = torch.zeros((8, 2, 2176), dtype=torch.uint8, device=DEV), torch.zeros((8, 2, 16), device=DEV)
        da.decode_attn_paged_fp8_weights(q, None, None, kv, w, torch.zeros((2, 4), dtype=torch.int32, device=DEV), sl, None, 0,
                                         0.125, torch.empty_like(q), scale_rule=2)
    assert e.value.code == -1
