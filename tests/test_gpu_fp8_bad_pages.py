"""A block-table entry outside the pool, on an fp8 cache: the tile reads zeros (16 keys of score 0 and value 0), as the
header states for every paged call, and never another sequence's block. Against the fp64 oracle with a
block of zero codes and zero scales in the entry's place; block 0, which nobody owns, holds NaN."""
import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
from cases import make_case, paged_identity, shuffle_pages
from test_gpu_decode import DEV, assert_close, dev, dev_bits
from test_gpu_fp8 import pre, to_dev
from test_oracle_multi import Multi
from test_oracle_multi_fp8 import fp8_paged

pytestmark = pytest.mark.gpu


def pools(cache, bt):
    """The cache behind a block of NaN, as the call gets it, and with a block of zeros at its end, as the oracle reads it."""
    nan, zero = np.full_like(cache.blocks[:1], 0xFF), np.zeros_like(cache.blocks[:1])
    mine = oracle.Fp8Cache(np.concatenate([nan, cache.blocks]))
    return mine, oracle.Fp8Cache(np.concatenate([mine.blocks, zero])), np.where(bt >= 0, bt + 1, bt).astype(np.int32)


def check(got, want):
    assert da.decode_attn_device_status() == da.DA_STATUS_BAD_PAGE
    assert_close(got, want, "pages outside the pool")


@pytest.mark.parametrize("T", [1, 2, 4, 16])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_several_tokens(T, entry):
    m = Multi(3000 + T, 16, 2, [100, 75, 230], [T, T, max(1, T - 1)], T)
    cache, bt, _ = fp8_paged(m, 1)
    cache, full, bt = pools(cache, bt)
    table, want = bt.copy(), bt.copy()
    for b, i in ((0, 0), (0, 2), (2, 5), (2, 6)):  # history pages
        table[b, i], want[b, i] = entry, cache.blocks.shape[0]
    for window in (0, 90):
        out = torch.empty((3, T, 16, 64), dtype=torch.bfloat16, device=DEV)
        da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), to_dev(cache), dev(table), dev(m.lens),
                                       dev(m.sinks), window, m.c.scale, out, q_lens=dev(m.n))
        ref = oracle.decode_multi_fp8(m.q, m.k_new, m.v_new, full, m.lens, m.sinks, window, m.c.scale, block_table=want, q_lens=m.n)
        check(out.double().cpu().numpy(), ref)


@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (16, 1)])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_one_token(Hq, Hkv, entry):
    c = make_case(3010, 3, Hq, Hkv, 64, [100, 75, 230])
    kp, vp, bt = shuffle_pages(*paged_identity(c, pre(c)), 1)
    cache = oracle.scatter_fp8(c.hist_k, c.hist_v, pre(c), oracle.Fp8Cache.empty_paged(kp.shape[0], Hkv, 16, 64), block_table=bt)
    cache, full, bt = pools(cache, bt)
    table, want = bt.copy(), bt.copy()
    for b, i in ((0, 0), (0, 2), (2, 5), (2, 6)):
        table[b, i], want[b, i] = entry, cache.blocks.shape[0]
    out = torch.empty((3, Hq, 64), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_fp8(dev_bits(c.q), dev_bits(c.k_new), dev_bits(c.v_new), to_dev(cache), dev(table), dev(c.lens), dev(c.sinks), 0,
                             c.scale, out)
    ref = oracle.decode_paged_fp8(c.q, c.k_new, c.v_new, full, want, c.lens, c.sinks, 0, c.scale)
    check(out.double().cpu().numpy(), ref)


@pytest.mark.parametrize("T", [4, 16])
@pytest.mark.parametrize("entry", [-2, -2 ** 31, 2 ** 31 - 1])
def test_every_entry_outside_the_pool_is_reported(T, entry):
    m = Multi(3020 + T, 16, 2, [100, 75], [T, T], T)
    cache, bt, _ = fp8_paged(m, 1)
    table = bt.copy()
    table[1, 2] = entry
    out = torch.empty((2, T, 16, 64), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), to_dev(cache), dev(table), dev(m.lens), None, 0,
                                   m.c.scale, out, q_lens=dev(m.n))
    assert da.decode_attn_device_status() == da.DA_STATUS_BAD_PAGE
    assert out.isfinite().all()
