"""GPU parity of the accumulated weights where the several-token kernels stage keys and query rows in
rings: more stages than a ring has slots, two key tiles per CTA, runs that end early, keys of pages
outside the pool in a reused slot, windows that begin inside a CTA's keys. Each call against the
plain 64-bit form, within the bound of plain_weights.weights_tolerance, and its output against the
call without weights, bit for bit."""
import numpy as np
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
import plain_weights as pw
from cases import bf16_to_f64
from test_gpu_decode import DEV, dev, dev_bits
from test_gpu_weights import check_weights, logical, start_weights
from test_oracle_multi import Multi

pytestmark = pytest.mark.gpu


def run(m, window=0, sinks=True, q_lens=True, width=None, bad=()):
    """One several-token call. width: columns of the block table (the kernels divide their work by the
    longest sequence it could hold). bad: (sequence, table column) entries outside the pool; their
    tokens are attended as zeros and get no weight."""
    c = m.c
    kp, vp, bt = m.paged(1, table_width=width)
    w0 = start_weights(kp.shape[0], c.Hkv, bt, m.base, 1)
    table = bt.copy()
    for i, (b, col) in enumerate(bad):
        table[b, col] = -1 if i % 2 else kp.shape[0]
    kd, vd, k2, v2, w = dev_bits(kp), dev_bits(vp), dev_bits(kp), dev_bits(vp), dev(w0)
    q, kn, vn, sk = dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), dev(m.sinks) if sinks else None
    out, ref = (torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ql = dev(m.n) if q_lens else None
    da.decode_attn_paged_multi_weights(q, kn, vn, kd, vd, w, dev(table), dev(c.lens), sk, window, c.scale, out, q_lens=ql)
    da.decode_attn_paged_multi(q, kn, vn, k2, v2, dev(table), dev(c.lens), sk, window, c.scale, ref, q_lens=ql)
    assert da.decode_attn_device_status() == (da.DA_STATUS_BAD_PAGE if bad else 0)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    for a, b in ((kd, k2), (vd, v2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    keys, values = logical(c, c.lens)
    sk64, q64, got = m.sinks.astype(np.float64) if sinks else None, bf16_to_f64(m.q), w.cpu().numpy()
    for b, col in bad:
        for x in (keys, values):
            x[b][col * 16:col * 16 + 16] = 0
    for b, col in bad:  # left as they were; then as the check below expects the cells it visits
        np.testing.assert_array_equal(got[bt[b, col]].view(np.uint32), w0[bt[b, col]].view(np.uint32))
        L = int(c.lens[b])
        _, mass, seen = pw.step(q64[b], keys[b], values[b], L, int(m.n[b]), sk64, window, c.scale)
        for j in range(col * 16, col * 16 + 16):
            if seen[j]:
                got[bt[b, col], :, j % 16] += mass[j].astype(np.float32)
    check_weights(got, w0, bt, c.lens, m.n, q64, keys, values, sk64, window, c.scale)


# Keys stream past up to 256 query rows: a CTA's run of 128-key stages is a share of what the block
# table could hold (up to 16 stages), and a ring holds 3 (32 rows), 4 (64, 128) or 8 (256) of them.
@pytest.mark.parametrize("T", [4, 8, 16, 32])
@pytest.mark.parametrize("bad", [(), ((0, 40), (0, 71), (1, 5), (1, 66))])
def test_more_key_stages_than_the_ring_holds(T, bad):
    m = Multi(2000 + T, 64, 8, [5000, 2300, 1], [T, T - 1, 1], T)
    run(m, width=8192, bad=bad)
    run(m, width=8192, sinks=False, window=70000)


@pytest.mark.parametrize("Hq,T", [(64, 32), (1024, 16)])
def test_key_stages_behind_a_window(Hq, T):
    """Runs of the longest range a window leaves; the first stage of a sequence starts mid-tile."""
    m = Multi(2010 + T, Hq, 64, [5500, 4990], [T, T - 3], T)
    run(m, window=4859)


# Query rows stream past the keys (more than 256 rows): 256 keys per CTA where that still gives every
# SM one, else 128.
@pytest.mark.parametrize("Hq,Hkv,T,lens", [(64, 8, 64, [6000, 300]), (16, 1, 33, [40000, 12]), (8, 8, 300, [3000, 1007, 299]),
                                           (64, 8, 130, [2900, 130])])
def test_rows_past_two_key_tiles(Hq, Hkv, T, lens):
    """The last block of keys holds fewer than 128 of its 256 (6000 = 23 * 256 + 112) or ends in its
    second half; counts ragged, and several row blocks more than the ring of rows has slots."""
    n = [min(T, L) for L in lens]
    n[-1] = max(1, n[-1] // 2 + 3)
    m = Multi(2020 + T, Hq, Hkv, lens, n, T)
    run(m, width=4096)
    run(m, width=4096, sinks=False, bad=((0, 20), (0, 33)))


@pytest.mark.parametrize("window", [2817, 3001])
def test_rows_past_two_key_tiles_behind_a_window(window):
    m = Multi(2030 + window, 64, 8, [6000, 2900, 64], [64, 37, 64], 64)
    run(m, window=window)


def test_rows_past_two_key_tiles_of_a_long_chunk():
    """512 tokens of 8 heads: 32 blocks of 128 rows past every block of keys that all of them see."""
    run(Multi(2040, 64, 8, [4500, 513], [512, 511], 512), width=2048)


@pytest.mark.parametrize("T", [3, 8, 16, 64])
def test_every_count_implicit(T):
    """No q_lens and no window: every sequence has T new tokens."""
    run(Multi(2050 + T, 64, 8, [T, 5 * T + 7, 3000], [T] * 3, T), q_lens=False)
