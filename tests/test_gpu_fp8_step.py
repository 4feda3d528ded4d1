"""An engine's steps over an fp8 cache, as they follow one another: packed projections normed and rotated
(positions of three axes, not L - 1), prompts in chunks and drafts to verify through the several-token
call, one token through decode_attn_paged_fp8, the cache read back for code that wants bf16. Every output
and every cache byte against the oracle, fed with the rotated rows the calls made."""
import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
from paged_decode_attention_kv_gb300 import workloads as wl
from test_gpu_decode import DEV, assert_close, dev
from test_gpu_fp8 import assert_blocks_equal, from_dev, to_dev
from test_gpu_fp8_store import check_read
from test_gpu_qk_norm_rope import axis_of, check, packed, plain, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (8, 4)])
def test_prompt_drafts_and_decode(Hq, Hkv):
    B, width, sections = 3, 12, (12, 10, 10)
    pages = B * width + 2
    rng = np.random.default_rng(Hq)
    table = rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)
    cache = oracle.Fp8Cache.empty_paged(pages, Hkv, 16, 64)
    kv, bt = to_dev(cache), dev(table)
    cos, sin = tables(512)
    sinks = dev(rng.standard_normal(Hq).astype(np.float32))
    lens = np.zeros(B, np.int32)
    for step, T in enumerate([40, 70, 4, 4, 1, 1, 3]):
        n = np.array([T, max(1, T - 3 * step % T) if T > 1 else 1, T if step != 1 else 0], np.int32)
        lens = lens + n
        x, q, k, v, (wq, wk), g = packed(B * T, Hq, Hkv, 100 * step + Hq)
        pos = torch.randint(0, 512, (3, B * T), generator=g, device=DEV, dtype=torch.int32)
        qr, kr, vr = (torch.empty((B, T, h, 64), dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
        da.qk_norm_rope(q, k, pos, cos, sin, qr.view(-1, Hq, 64), kr.view(-1, Hkv, 64), q_weight=wq,
                        k_weight=wk, sections=sections, interleaved=True, v=v, v_out=vr.view(-1, Hkv, 64))
        check(kr.view(-1, Hkv, 64), *plain(k, pos, cos, sin, wk, 1e-6, axis_of(sections, True)))
        out = torch.empty((B, T, Hq, 64), dtype=torch.bfloat16, device=DEV)
        if T == 1:
            da.decode_attn_paged_fp8(qr[:, 0], kr[:, 0], vr[:, 0], kv, bt, dev(lens), sinks, 0, wl.SCALE, out[:, 0])
        else:
            da.decode_attn_paged_fp8_multi(qr, kr, vr, kv, bt, dev(lens), sinks, 0, wl.SCALE, out, q_lens=dev(n))
        bits = [wl.bits(y.cpu()) for y in (qr, kr, vr)]
        want = oracle.decode_multi_fp8(*bits, cache, lens, sinks.cpu().numpy(), 0, wl.SCALE, block_table=table, q_lens=n)
        assert_close(out.double().cpu().numpy(), want, f"step {step} of {T}")
        cache = oracle.kv_append_multi_fp8(bits[1], bits[2], cache, lens, block_table=table, q_lens=n)
        assert_blocks_equal(from_dev(kv), cache)
    assert da.decode_attn_device_status() == 0
    check_read(kv, cache, lens, int(lens.max()), table, starts=np.array([0, 17, 5], np.int32))


def test_nothing_to_do():
    """No token, no sequence, no row to read: every call returns, and the cache stays as it is."""
    def rows(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    cos, sin = tables(16)
    da.qk_norm_rope(rows(0, 8, 64), rows(0, 2, 64), torch.empty(0, dtype=torch.int32, device=DEV), cos, sin, rows(0, 8, 64), rows(0, 2, 64),
                    v=rows(0, 2, 64), v_out=rows(0, 2, 64))
    da.qk_norm_rope(rows(0, 8, 64), rows(0, 2, 64), torch.empty((3, 0), dtype=torch.int32, device=DEV), cos, sin, rows(0, 8, 64),
                    rows(0, 2, 64), sections=(12, 10, 10))
    kv = torch.randint(0, 120, (4, 2, da.FP8_BLOCK_BYTES), dtype=torch.uint8, device=DEV)
    before = kv.clone()
    sinks = torch.zeros(8, device=DEV)
    table, lens = torch.zeros((0, 4), dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    da.kv_append_fp8(rows(0, 5, 2, 64), rows(0, 5, 2, 64), kv, lens, block_table=table)
    da.kv_append_fp8(rows(0, 5, 2, 64), rows(0, 5, 2, 64), kv[:0].view(0, 2, 1, da.FP8_BLOCK_BYTES), lens)
    da.kv_read_fp8(kv, lens, rows(0, 7, 2, 64), rows(0, 7, 2, 64), block_table=table)
    for T in (2, 40):
        da.decode_attn_paged_fp8_multi(rows(0, T, 8, 64), rows(0, T, 2, 64), rows(0, T, 2, 64), kv, table, lens, sinks, 0, 0.125, rows(0, T, 8, 64))
    table, lens = torch.zeros((2, 4), dtype=torch.int32, device=DEV), torch.tensor([9, 0], dtype=torch.int32, device=DEV)
    da.kv_read_fp8(kv, lens, rows(2, 0, 2, 64), rows(2, 0, 2, 64), block_table=table)
    torch.cuda.synchronize()
    assert da.decode_attn_device_status() == 0 and torch.equal(kv, before)
