"""GPU parity of kv_append_fp8 and kv_read_fp8: the appended blocks byte for byte against the oracle's
quantised append (every byte of every block: what is not appended stays as it was), the rows read back
bit for bit against code value * scale in fp32 rounded to bf16, and rows past them left as they were."""
import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
from paged_decode_attention_kv_gb300 import workloads as wl
from test_gpu_decode import DEV, dev, dev_bits
from test_gpu_fp8 import assert_blocks_equal, from_dev, to_dev
from test_gpu_multi import LENS, counts
from test_oracle_multi import Multi
from test_oracle_multi_fp8 import fp8_paged

pytestmark = pytest.mark.gpu


def ring_of(m, W):
    return oracle.scatter_fp8(m.c.hist_k, m.c.hist_v, m.base, oracle.Fp8Cache.empty_ring(m.c.B, m.c.Hkv, W, 64), window=W)


def check_append(m, blocks, bt=None, W=0, q_lens=True, **kw):
    kv = to_dev(blocks)
    da.kv_append_fp8(dev_bits(m.k_new), dev_bits(m.v_new), kv, dev(m.lens), None if bt is None else dev(bt),
                     q_lens=dev(m.n) if q_lens else None, **kw)
    assert da.decode_attn_device_status() == 0
    want = oracle.kv_append_multi_fp8(m.k_new, m.v_new, blocks, m.lens, block_table=bt, window=W, q_lens=m.n if q_lens else None)
    assert_blocks_equal(from_dev(kv), want)
    return kv, want


def cells(cache, bt, W, b, pos):
    """fp32 K and V rows [len(pos), Hkv, 64] of positions pos of sequence b."""
    k, v = [], []
    for p in pos:
        blk = (bt[b, p // 16],) if bt is not None else (b,)
        i = (slice(None),) if bt is not None else (slice(None), p % W // 16)
        at = blk + i
        k.append(oracle.e4m3_decode(cache.k[at][:, p % 16]).astype(np.float32) * cache.ks[at][:, p % 16][:, None])
        v.append(oracle.e4m3_decode(cache.vt[at][:, :, p % 16]).astype(np.float32) * cache.vs[at][:, p % 16][:, None])
    return (np.stack(k), np.stack(v)) if len(pos) else (np.zeros((0, cache.k.shape[1], 64), np.float32),) * 2


def check_read(kv, cache, lens, rows, bt=None, W=0, starts=None, **kw):
    B, Hkv = len(lens), cache.k.shape[1]
    k, v = (torch.full((B, rows, Hkv, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    da.kv_read_fp8(kv, dev(lens), k, v, None if bt is None else dev(bt), starts=None if starts is None else dev(starts), **kw)
    assert da.decode_attn_device_status() == 0
    for b, L in enumerate(lens):
        first = 0 if starts is None else int(starts[b])
        n = max(0, min(int(L) - first, rows))
        for got, want in zip((k, v), cells(cache, bt, W, b, range(first, first + n))):
            np.testing.assert_array_equal(wl.bits(got[b, :n].cpu()), wl.bits(torch.from_numpy(want).to(torch.bfloat16)))
            assert (got[b, n:] == 7).all()


@pytest.mark.parametrize("Hkv", [8, 1, 3])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 40, 257])
def test_paged(Hkv, T):
    m = Multi(2100 + Hkv + T, 2 * Hkv, Hkv, LENS, counts(T, LENS, Hkv + T), T)
    blocks, bt, _ = fp8_paged(m, T)
    kv, want = check_append(m, blocks, bt)
    lens = m.lens
    rows = int(lens.max())
    check_read(kv, want, lens, rows, bt)
    check_read(kv, want, lens, rows, bt, starts=m.base)
    check_read(kv, want, lens, 5, bt, starts=np.minimum(lens, 13).astype(np.int32))
    check_read(kv, want, lens, rows + 33, bt, max_seq_len=rows)


@pytest.mark.parametrize("W", [16, 128])
@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_ring(W, T):
    lens = [1, 15, 16, 17, W - 1, W, W + 1, 3 * W + 5, 60, 0]
    m = Multi(2200 + W + T, 8, 4, lens, counts(T, lens, W + T), T)
    kv, want = check_append(m, ring_of(m, W), W=W)
    check_read(kv, want, m.lens, W, W=W, starts=np.maximum(m.lens - W, 0).astype(np.int32))
    check_read(kv, want, m.lens, 7, W=W, starts=np.maximum(m.lens - 5, 0).astype(np.int32))


def test_one_token_rows_and_no_counts():
    """k_new of [B, Hkv, 64], as the one-token calls take it, and T tokens of every sequence."""
    m = Multi(2300, 8, 4, [3, 16, 17], [1, 1, 1], 1)
    blocks, bt, _ = fp8_paged(m, 1)
    kv = to_dev(blocks)
    da.kv_append_fp8(dev_bits(m.k_new[:, 0].copy()), dev_bits(m.v_new[:, 0].copy()), kv, dev(m.lens), dev(bt))
    assert_blocks_equal(from_dev(kv), oracle.kv_append_fp8(m.k_new[:, 0], m.v_new[:, 0], blocks, m.lens, block_table=bt))
    m = Multi(2301, 8, 4, [30, 16, 17], [13] * 3, 13)
    blocks, bt, _ = fp8_paged(m, 1)
    check_append(m, blocks, bt, q_lens=False)


def test_rows_of_every_kind():
    """Rows of zeros, of the smallest and the largest magnitudes, exact ties of e4m3, and every bf16
    mantissa against scales of many sizes: the oracle's codes."""
    m = Multi(2310, 4, 4, [512], [512], 512)
    rng = np.random.default_rng(3)
    x = rng.integers(0, 1 << 16, (512, 4, 64)).astype(np.uint16)
    x[(x & 0x7F80) == 0x7F80] &= 0x3FFF                       # every finite value
    near = rng.integers(0x3C00, 0x4380, (256, 4, 64)).astype(np.uint16) | (rng.integers(0, 2, (256, 4, 64)) << 15).astype(np.uint16)
    x[:256] = near                                             # values of one row within a few powers of two
    x[5] = 0
    x[6] = 0x8000                                              # negative zeros
    x[7] = 1                                                   # the smallest magnitude
    x[8, :, 1:] = 0x3F80
    x[8, :, 0] = 0x43E0                                        # 448: the scale is 1, codes on the grid
    x[9] = x[8]
    x[9, :, 1:] = (0x3F84 + 8 * np.arange(63) % 64).astype(np.uint16)   # 1 + (odd) / 32 ...: ties among them
    x[10] = 0x7F7F                                             # the largest
    m.k_new, m.v_new = x[None].copy(), np.roll(x, 3, axis=0)[None].copy()
    blocks, bt, _ = fp8_paged(m, 1)
    check_append(m, blocks, bt)
    check_append(m, ring_of(m, 512), W=512)


@pytest.mark.parametrize("ring", [False, True])
def test_bad_sequences_are_left_alone(ring):
    m = Multi(2320, 4, 2, [60, 60, 60, 60], [20] * 4, 20)
    W = 64
    blocks, bt, _ = fp8_paged(m, 1)
    if ring:
        blocks, bt = ring_of(m, W), None
    lens, n = m.lens.copy(), m.n.copy()
    lens[1], n[2] = -1, 21
    table = None
    if not ring:
        table = bt.copy()
        table[3, 2] = blocks.blocks.shape[0]                   # positions 32 .. 47: 40 .. 47 are new
    kv = to_dev(blocks)
    da.kv_append_fp8(dev_bits(m.k_new), dev_bits(m.v_new), kv, dev(lens), None if ring else dev(table), q_lens=dev(n))
    want = oracle.kv_append_multi_fp8(m.k_new, m.v_new, blocks, m.lens, block_table=bt, window=W if ring else 0,
                                      q_lens=np.array([20, 0, 0, 20], np.int32))
    if not ring:  # the tokens of the bad page are skipped
        want.blocks[bt[3, 2]] = blocks.blocks[bt[3, 2]]
    status = da.DA_STATUS_BAD_SEQ_LEN | (0 if ring else da.DA_STATUS_BAD_PAGE)
    assert da.decode_attn_device_status() == status
    assert_blocks_equal(from_dev(kv), want)
    # read back: the bad ones' rows stay, a page outside the pool leaves its rows
    k, v = (torch.full((4, 64, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    starts = np.array([0, 0, 61, 0], np.int32)
    da.kv_read_fp8(kv, dev(lens), k, v, None if ring else dev(table), starts=dev(starts))
    assert da.decode_attn_device_status() == status
    assert (k[1:3] == 7).all() and (v[1:3] == 7).all() and (k[0, :60] != 7).any() and (k[3, 60:] == 7).all()
    if not ring:
        assert (k[3, 32:48] == 7).all() and (v[3, 32:48] == 7).all()


def test_positions_that_a_ring_dropped():
    m = Multi(2330, 4, 2, [60], [20], 20)
    kv = to_dev(ring_of(m, 32))
    k, v = (torch.zeros((1, 64, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    da.kv_read_fp8(kv, dev(m.lens), k, v, starts=dev(np.array([27], np.int32)))
    assert da.decode_attn_device_status() == da.DA_STATUS_BAD_SEQ_LEN and not k.any()


def test_outputs_at_16_bytes():
    """Rows at a 16-byte address that is not a 32-byte one."""
    m = Multi(2340, 4, 2, [50, 3], [7, 3], 7)
    blocks, bt, _ = fp8_paged(m, 1)
    kv, want = check_append(m, blocks, bt)
    n = 2 * 50 * 2 * 64
    k, v = (torch.zeros(n + 8, dtype=torch.bfloat16, device=DEV)[8:].view(2, 50, 2, 64) for _ in range(2))
    da.kv_read_fp8(kv, dev(m.lens), k, v, dev(bt))
    full, _ = cells(want, bt, 0, 0, range(50))
    np.testing.assert_array_equal(wl.bits(k[0].cpu()), wl.bits(torch.from_numpy(full).to(torch.bfloat16)))
