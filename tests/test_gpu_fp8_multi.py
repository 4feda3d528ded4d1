"""GPU parity of the several-token step over an fp8 cache (decode_attn_paged_fp8_multi) against
the fp64 oracle over the same codes and scales, the new tokens attended as they are stored:
every output row within 4e-3 + 1e-2 |oracle| (rows beyond q_lens and inactive slots exactly zero),
every byte of the cache after the call. Dead cells, and the padding rows of k_new / v_new, hold NaN
codes, NaN scales and NaN, so reading any of them shows.

The bar, for inputs of unit variance: bf16's half step 2^-8 of the output; fp16's half steps 2^-11 on
the probabilities and on the cached values; and on the scores 0.125 sqrt(64) 2^-11 / sqrt(3) for their
standard deviation, twice that on a probability's ratio to the others: all below 1e-2 relative."""
import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
from test_gpu_decode import DEV, assert_close, dev, dev_bits
from test_gpu_fp8 import assert_blocks_equal, from_dev, to_dev
from test_gpu_multi import LENS, counts
from test_oracle_multi import Multi
from test_oracle_multi_fp8 import fp8_paged

pytestmark = pytest.mark.gpu


def run(m, window, seed=1, q_lens=True, sinks=True, cache=None, **kw):
    """One call checked against the oracle; returns its output."""
    blocks, bt, _ = fp8_paged(m, seed)
    if cache is not None:
        cache(blocks)
    kv, c = to_dev(blocks), m.c
    out = torch.full((c.B, m.T, c.Hq, c.D), float("nan"), dtype=torch.bfloat16, device=DEV)
    n = dev(m.n) if q_lens else None
    da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), kv, dev(bt), dev(m.lens),
                                   dev(m.sinks) if sinks else None, window, c.scale, out, q_lens=n, **kw)
    torch.cuda.synchronize()
    assert da.decode_attn_device_status() == 0
    n = m.n if q_lens else None
    ref = oracle.decode_multi_fp8(m.q, m.k_new, m.v_new, blocks, m.lens, m.sinks if sinks else None, window, c.scale,
                                  block_table=bt, q_lens=n)
    assert_close(out.double().cpu().numpy(), ref, f"fp8 multi window={window}")
    for b in range(c.B):
        assert not out[b, int(m.n[b]):].any()
    assert_blocks_equal(from_dev(kv), oracle.kv_append_multi_fp8(m.k_new, m.v_new, blocks, m.lens, block_table=bt, q_lens=n))
    return out


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (8, 8), (16, 1), (32, 4), (6, 3)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 9, 16, 40])
@pytest.mark.parametrize("window", [0, 7, 100])
def test_matches_oracle(Hq, Hkv, T, window):
    """Up to 4 tokens and 32 query rows per KV head (8, 16 and 32 of them) in the decode kernel, more on
    tcgen05: one row block, part of one, several."""
    m = Multi(1800 + Hq + T + window, Hq, Hkv, LENS, counts(T, LENS, Hq + T + window), T)
    run(m, window, seed=T + 1)


@pytest.mark.parametrize("T", [4, 16])
def test_long_sequences_and_splits(T):
    lens = [5000, 12001, 131, T]
    m = Multi(1900 + T, 64, 8, lens, [T, T, 3, T], T)
    run(m, 0)
    run(m, 4001, sinks=False)
    run(m, 0, max_seq_len=12001)


def test_one_long_sequence_over_every_cta():
    for T in (2, 17):
        m = Multi(1910 + T, 16, 2, [40000], [T], T)
        run(m, 0)


@pytest.mark.parametrize("Hq,Hkv,T", [(64, 8, 130), (16, 1, 100), (4, 4, 300)])
def test_prompts(Hq, Hkv, T):
    """Whole prompts and chunks of them: many row blocks, whose last rows are not queries."""
    lens = [T, T + 77, 1, 64, 500, 0]
    m = Multi(1920 + T, Hq, Hkv, lens, [min(L, T) for L in lens], T)
    run(m, 0)
    run(m, 50)


def test_without_q_lens_and_without_sinks():
    for T in (3, 12):
        m = Multi(1930 + T, 32, 4, [T, 40, 100], [T] * 3, T)
        run(m, 0, q_lens=False)
        run(m, 0, sinks=False)


def test_rows_without_keys_or_sequences():
    """No new token anywhere, and no active slot: zeros, and an untouched cache."""
    for T in (4, 8):
        m = Multi(1940 + T, 8, 1, [5, 20, 0], [0, 0, 0], T)
        run(m, 0)
        run(Multi(1945, 8, 1, [0, 0], [0, 0], T), 0, sinks=False)


def test_one_new_token_is_the_one_token_step():
    m = Multi(1950, 64, 8, [1, 16, 17, 300], [1] * 4, 1)
    out = run(m, 0)
    blocks, bt, _ = fp8_paged(m, 1)
    one = torch.empty_like(out[:, 0])
    kv = to_dev(blocks)
    da.decode_attn_paged_fp8(dev_bits(m.q[:, 0].copy()), dev_bits(m.k_new[:, 0].copy()), dev_bits(m.v_new[:, 0].copy()), kv, dev(bt), dev(m.lens),
                             dev(m.sinks), 0, m.c.scale, one)
    # the same fp16 products in another order, each output rounded to bf16
    assert (one.float() - out[:, 0].float()).abs().max() <= 2 * 2.0 ** -8 * one.float().abs().max()


@pytest.mark.parametrize("T", [4, 24])
def test_scales_of_very_different_size(T):
    """Tokens whose K and V scales differ by powers of two, within pages and between them. The V
    values span 2^-30 .. 2^9, so the error is measured against the probability-weighted magnitudes:
    P and V' each off by fp16's half step of the page's largest factor, the output by bf16's, the
    scores (at most 2^3 in magnitude here) by 2^3 2^-11 twice over."""
    m = Multi(1960 + T, 16, 2, [200, 77, 1000], [T] * 3, T)
    rng = np.random.default_rng(5)
    blocks, bt, _ = fp8_paged(m, 1)
    live = np.isfinite(blocks.ks)
    blocks.ks[...] = np.where(live, blocks.ks * 2.0 ** rng.integers(-12, 1, blocks.ks.shape), blocks.ks)
    blocks.vs[...] = np.where(live, blocks.vs * 2.0 ** rng.integers(-30, 1, blocks.vs.shape), blocks.vs)
    big = rng.integers(0, 2, blocks.vs.shape[0]) == 1  # half of the pages 2^9 larger
    blocks.vs[big] *= 512
    kv = to_dev(blocks)
    out = torch.empty((3, T, 16, 64), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), kv, dev(bt), dev(m.lens),
                                   dev(m.sinks), 0, m.c.scale, out, q_lens=dev(m.n))
    args = (m.lens, m.sinks, 0, m.c.scale)
    ref = oracle.decode_multi_fp8(m.q, m.k_new, m.v_new, blocks, *args, block_table=bt, q_lens=m.n)
    mag = blocks.copy()
    mag.vt[...] &= 0x7F
    vabs = (m.v_new & 0x7FFF).astype(np.uint16)
    weight = oracle.decode_multi_fp8(m.q, m.k_new, vabs, mag, *args, block_table=bt, q_lens=m.n)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + (2 * 2.0 ** -11 + 2 * 2.0 ** -8) * weight).all()


@pytest.mark.parametrize("power", [-40, 40])
def test_values_far_from_one(power):
    """V of 2^-40 and 2^40 give the digits of V of 1: probabilities, operands and sums are the same numbers but for a power
    of two; only the division at the end, where the sink joins, rounds in fp32 elsewhere, so that an output may land on
    bf16's next value: two half steps. On tcgen05; the decode kernel's fp16 products hold scales of ordinary size."""
    m = Multi(1970, 16, 2, [200, 77], [16, 5], 16)
    plain = run(m, 0).float()
    blocks, bt, _ = fp8_paged(m, 1)
    blocks.vs[...] *= np.float32(2.0 ** power)
    v = (torch.from_numpy(m.v_new.view(np.int16)).view(torch.bfloat16).float() * 2.0 ** power).to(torch.bfloat16)
    out = torch.empty((2, 16, 16, 64), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), v.to(DEV), to_dev(blocks), dev(bt), dev(m.lens), dev(m.sinks),
                                   0, m.c.scale, out, q_lens=dev(m.n))
    assert ((out.float() * 2.0 ** -power - plain).abs() <= 2 * 2.0 ** -8 * plain.abs()).all()


def test_sharp_softmax():
    """Scores up to a few hundred: one key takes all of a row, references move often. The K operand's
    fp16 rounding moves a score s by at most |s| 2^-11, so rows are compared where the winner leads."""
    m = Multi(1980, 16, 2, [400, 90], [20, 20], 20)
    m.q = (m.q.astype(np.uint32) + (4 << 7)).astype(np.uint16)  # 16 times as large
    blocks, bt, _ = fp8_paged(m, 1)
    out = torch.empty((2, 20, 16, 64), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), to_dev(blocks), dev(bt), dev(m.lens), None,
                                   0, m.c.scale, out, q_lens=dev(m.n))
    ref = oracle.decode_multi_fp8(m.q, m.k_new, m.v_new, blocks, m.lens, None, 0, m.c.scale, block_table=bt, q_lens=m.n)
    # scores of standard deviation 16: |s| below 100, moved by 100 2^-11 at most, so a probability by e^0.05 - 1
    # twice over, times values of at most 4.5
    err = np.abs(out.double().cpu().numpy() - ref)
    assert err.max() <= 2 * 0.0513 * 4.5
    assert np.median(err) <= 2.0 ** -8


def test_a_prompt_in_chunks_is_the_whole_prompt():
    """The same cache bit for bit, and the same outputs but for the order of the sums."""
    L, cut = 300, 16
    m = Multi(1990, 64, 8, [L], [L], L)
    whole = run(m, 0)
    blocks, bt, _ = fp8_paged(m, 1)
    kv, outs = to_dev(blocks), []
    for at in range(0, L, cut):
        n = min(cut, L - at)
        out = torch.empty((1, n, 64, 64), dtype=torch.bfloat16, device=DEV)
        da.decode_attn_paged_fp8_multi(dev_bits(m.q[:, at:at + n].copy()), dev_bits(m.k_new[:, at:at + n].copy()), dev_bits(m.v_new[:, at:at + n].copy()),
                                       kv, dev(bt), dev(np.array([at + n], np.int32)), dev(m.sinks), 0, m.c.scale, out)
        outs.append(out)
    parts = torch.cat(outs, 1).float()
    assert ((parts - whole.float()).abs() <= 2 * 2.0 ** -8 * whole.float().abs() + 2e-3).all()
    assert_blocks_equal(from_dev(kv), oracle.kv_append_multi_fp8(m.k_new, m.v_new, blocks, m.lens, block_table=bt, q_lens=m.n))


@pytest.mark.parametrize("T", [4, 16])
def test_scale_rules(T):
    m = Multi(2000 + T, 16, 2, [T, 50], [T, T], T)
    blocks, bt, _ = fp8_paged(m, 1)
    got = []
    for rule in (da.DA_FP8_SCALE_DIVIDE, da.DA_FP8_SCALE_RECIPROCAL):
        kv = to_dev(blocks)
        out = torch.empty((2, T, 16, 64), dtype=torch.bfloat16, device=DEV)
        da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), kv, dev(bt), dev(m.lens), None, 0, m.c.scale, out,
                                       scale_rule=rule)
        got.append(from_dev(kv))
        top = np.abs((m.v_new[0].astype(np.uint32) << 16).view(np.float32)).max(-1)     # [T, Hkv]
        want = (top / np.float32(448) if rule == da.DA_FP8_SCALE_DIVIDE else top * np.float32(1 / 448)).astype(np.float32)
        np.testing.assert_array_equal(got[-1].vs[bt[0, 0], :, :min(T, 16)].T, want[:16])
    assert (got[0].blocks != got[1].blocks).any()


@pytest.mark.parametrize("T", [4, 16])
def test_bad_lengths_and_pages(T):
    """A bad count or length makes its slot inactive, a page outside the pool reads zeros (decode kernel: another
    block) and takes no append; the other slots are as without them."""
    m = Multi(2010 + T, 16, 2, [60, 60, 60, 60], [T] * 4, T)
    ok = run(m, 0)
    blocks, bt, _ = fp8_paged(m, 1)
    lens, n, table = m.lens.copy(), m.n.copy(), bt.copy()
    lens[1] = bt.shape[1] * 16 + 1
    n[2] = T + 1
    table[3, 0] = blocks.blocks.shape[0]
    kv = to_dev(blocks)
    out = torch.full((4, T, 16, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_fp8_multi(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), kv, dev(table), dev(lens), dev(m.sinks), 0, m.c.scale, out,
                                   q_lens=dev(n))
    assert da.decode_attn_device_status() == da.DA_STATUS_BAD_SEQ_LEN | da.DA_STATUS_BAD_PAGE
    assert torch.equal(out[0], ok[0]) and not out[1].any() and not out[2].any()
    after = oracle.kv_append_multi_fp8(m.k_new, m.v_new, blocks, m.lens, block_table=bt, q_lens=np.array([T, 0, 0, T], np.int32))
    assert_blocks_equal(from_dev(kv), after)


@pytest.mark.parametrize("T", [4, 16, 64])
def test_captured_calls_and_streams(T):
    """A captured call replayed with other lengths, at every early-input level, next to calls on another stream."""
    lens = [100, 300, 64]
    m = Multi(2020 + T, 64, 8, lens, [T] * 3, T)
    blocks, bt, _ = fp8_paged(m, 1)
    c = m.c
    kv, other = to_dev(blocks), to_dev(blocks)
    q, k, v, table, n, sinks = dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), dev(bt), dev(m.n), dev(m.sinks)
    sl = dev(m.lens)
    out, out2 = (torch.empty((3, T, 64, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    da.decode_attn_multi_reserve(da.decode_attn_paged_fp8_multi_workspace_bytes(3, 64, 8, T, 0, bt.shape[1] * 16))
    want = run(m, 0)
    graph, stream, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    da.decode_attn_stream_reserve(side)
    try:
        for level in (0, 1, 2):
            before = da.decode_attn_set_early_inputs(level)
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                da.decode_attn_paged_fp8_multi(q, k, v, kv, table, sl, sinks, 0, c.scale, out, q_lens=n)
                da.decode_attn_paged_fp8_multi(q, k, v, kv, table, sl, sinks, 0, c.scale, out, q_lens=n)
            da.decode_attn_set_early_inputs(before)
            sl.copy_(dev(np.array([0, 0, 0], np.int32)))
            graph.replay()
            torch.cuda.synchronize()
            assert not out.any()
            sl.copy_(dev(m.lens))
            torch.cuda.synchronize()
            graph.replay()
            with torch.cuda.stream(side):
                da.decode_attn_paged_fp8_multi(q, k, v, other, table, sl, sinks, 0, c.scale, out2, q_lens=n)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(out2, want)
        assert da.decode_attn_device_status() == 0
    finally:
        da.decode_attn_stream_release(side)


@pytest.mark.parametrize("lens", ["short", "units"])
def test_segments_far_from_one_another(lens):
    """Many short sequences whose scores lie up to 800 apart from one KV head to the next (the last element of every key
    is 16, exactly, in every form that it takes; the queries' says how far): nothing of one may be left to the next.
    A softmax does not change by what all of its scores share, so the bar is that of ordinary inputs."""
    B = 96 if lens == "short" else 40
    L = [17 + 13 * b % 50 for b in range(B)] if lens == "short" else [16 + 37 * b % 400 for b in range(B)]
    m = Multi(1995 + B, 64, 8, L, [16 - b % 3 for b in range(B)], 16)
    for hist in (m.c.hist_k, [m.k_new]):
        for k in hist:
            k[..., 63] = 0x4180  # 16 in bf16
    offset = np.array([0.0, 400.0, -400.0, 32.0, -4.0], np.float32)[(3 * np.arange(B)[:, None] + np.arange(8)[None, :]) % 5]
    m.q[..., 63] = np.repeat(offset.view(np.uint32) >> 16, 8, axis=1)[:, None, :].astype(np.uint16)
    run(m, 0, sinks=False)
    run(m, 40, sinks=False)
    run(m, 0)


def test_rows_without_a_reference_beside_rows_left_behind():
    """Behind a window of 70, tokens 32 .. 63 of 128 share a warp; the first keys are cut into 96 .. 159 and 160 .. 223. The
    last seven of the tokens see none of the first, the others a few, whose scores lie 300 below those of the second:
    all of them find their reference there at the same time."""
    L, T = 300, 128
    m = Multi(1998, 4, 4, [L, L, L], [T, T, T], T)
    for at in range(160, L):  # (the history is the first L - T)
        (m.c.hist_k[:, at] if at < L - T else m.k_new[:, at - (L - T)])[..., 63] = 0x4180  # 16
    for at in range(160):
        m.c.hist_k[:, at, :, 63] = 0
    m.q[..., 63] = 0x4316  # 150 in bf16: 0.125 * 16 * 150 = 300
    for window in (70, 75, 40, 0):
        run(m, window, sinks=False)
