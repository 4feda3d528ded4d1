"""Rows of zeros in an fp8 cache, on the tcgen05 route of decode_attn_paged_fp8_multi. A row of zeros has scale 1 by
the format, however small the rows around it are; it must cost the other tokens of its page, and the other
pages, no precision. Against the fp64 oracle over the same codes and scales.

The bar is measured against the probability-weighted magnitudes W = sum p_j |v_j| and does not know how large V is: an
output is rounded to bf16 (2^-8 of it), P once and V' twice to fp16 (3 x 2^-11 of W), and the scores, at most 2^3 in
magnitude, move by 2^3 2^-11 at most, twice over (2 x 2^-8 of W)."""
import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
from test_gpu_decode import DEV, dev, dev_bits
from test_gpu_fp8 import to_dev
from test_oracle_multi import Multi
from test_oracle_multi_fp8 import fp8_paged

pytestmark = pytest.mark.gpu


def scaled(bits, power):
    """bf16 bits times 2^power (exact for the normal values of these tests)."""
    x = (bits.astype(np.uint32) << 16).view(np.float32) * np.float32(2.0 ** power)
    return (x.view(np.uint32) >> 16).astype(np.uint16)


def set_rows(m, which, at, value):
    """Positions at(b) of K ("k") or V ("v") of every sequence, history and new tokens, set to `value`."""
    hist = m.c.hist_k if which == "k" else m.c.hist_v
    new = m.k_new if which == "k" else m.v_new
    for b in range(m.c.B):
        for p in at(b):
            if p < m.base[b]:
                hist[b, p] = value
            elif p < m.lens[b]:
                new[b, p - m.base[b]] = value


def check(m, window=0, sinks=True):
    blocks, bt, _ = fp8_paged(m, 1)
    out = torch.empty((m.c.B, m.T, m.c.Hq, 64), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), to_dev(blocks), dev(bt), dev(m.lens),
                                   dev(m.sinks) if sinks else None, window, m.c.scale, out, q_lens=dev(m.n))
    assert da.decode_attn_device_status() == 0
    args = (m.lens, m.sinks if sinks else None, window, m.c.scale)
    ref = oracle.decode_multi_fp8(m.q, m.k_new, m.v_new, blocks, *args, block_table=bt, q_lens=m.n)
    mag = blocks.copy()
    mag.vt[...] &= 0x7F
    weight = oracle.decode_multi_fp8(m.q, m.k_new, (m.v_new & 0x7FFF).astype(np.uint16), mag, *args, block_table=bt, q_lens=m.n)
    err = np.abs(out.double().cpu().numpy() - ref)
    bar = 2.0 ** -8 * np.abs(ref) + (3 * 2.0 ** -11 + 2 * 2.0 ** -8) * weight
    assert (err <= bar).all(), f"worst {np.nanmax(err / np.maximum(weight, 1e-300)):.3g} of the weighted magnitude"


@pytest.mark.parametrize("power", [-12, -16, -24])
@pytest.mark.parametrize("zero", [0x0000, 0x8000])
def test_zero_values_beside_small_ones(power, zero):
    """A row of (negative) zeros in every page of V far below 1."""
    m = Multi(2400, 16, 2, [16, 40, 90, 33], [16, 9, 16, 16], 16)
    m.c.hist_v[...] = scaled(m.c.hist_v, power)
    m.v_new[...] = scaled(m.v_new, power)
    set_rows(m, "v", lambda b: range(3 + b, 100, 16), zero)
    check(m)
    check(m, window=21, sinks=False)


@pytest.mark.parametrize("power", [-12, -24])
def test_pages_of_zero_values(power):
    """Whole pages of zeros in a long history of small values: they count in the denominators alone."""
    m = Multi(2410, 16, 2, [1500, 333], [16, 5], 16)
    m.c.hist_v[...] = scaled(m.c.hist_v, power)
    m.v_new[...] = scaled(m.v_new, power)
    set_rows(m, "v", lambda b: range(320, 336), 0)
    set_rows(m, "v", lambda b: range(16, 48), 0)
    check(m)
    check(m, sinks=False)


def test_zero_keys_beside_small_ones():
    """Rows of zeros in K far below 1, under queries as much larger."""
    m = Multi(2420, 16, 2, [16, 40, 90, 200], [16, 9, 16, 16], 16)
    m.c.hist_k[...] = scaled(m.c.hist_k, -13)
    m.k_new[...] = scaled(m.k_new, -13)
    m.q[...] = scaled(m.q, 13)
    set_rows(m, "k", lambda b: range(5 + b, 200, 16), 0)
    set_rows(m, "k", lambda b: range(7 + b, 200, 32), 0x8000)
    check(m)


def test_rows_of_scale_one_that_are_not_zeros():
    """Values whose largest magnitude is 448 have scale 1 too, and so have zeros beside them."""
    m = Multi(2430, 16, 2, [60, 37], [16, 16], 16)
    for x in (m.c.hist_v, m.v_new):
        x[..., 0] = 0x43E0                                      # 448
    set_rows(m, "v", lambda b: range(2 + b, 60, 7), 0)
    set_rows(m, "v", lambda b: range(4, 60, 11), 0x0080)        # 2^-126: codes of no common size with the others'
    check(m)


def test_only_zeros():
    m = Multi(2440, 16, 2, [60, 300], [16, 16], 16)
    set_rows(m, "v", lambda b: range(0, 300), 0)
    set_rows(m, "k", lambda b: range(0, 300), 0)
    check(m)
    check(m, sinks=False)
