"""GPU parity of the calls that accumulate attention weights (decode_attn_paged_weights, _fp8_weights,
_multi_weights) against the plain 64-bit form: every weight cell within the bound derived in
plain_weights.weights_tolerance, cells that were not attended bit-unchanged (dead cells hold NaN,
in the caches and in the weights), the output and the caches as the call without weights gives
them, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
import plain_weights as pw
from cases import bf16_to_f64, paged_identity, shuffle_pages
from paged_decode_attention_kv_gb300 import workloads as wl
from test_gpu_decode import DEV, assert_close, dev, dev_bits
from test_gpu_multi import counts, ramp_keys
from test_oracle_multi import Multi

pytestmark = pytest.mark.gpu


def start_weights(pool_pages, Hkv, bt, base, seed):
    """Weights of the history's cells, NaN everywhere else."""
    rng = np.random.default_rng(seed)
    w = np.full((pool_pages, Hkv, 16), np.nan, np.float32)
    for b, L in enumerate(base):
        c = np.arange(L)
        w[bt[b, c // 16], :, c % 16] = rng.exponential(size=(L, Hkv)).astype(np.float32) ** 3
    return w


def check_weights(got, w0, bt, lens, n, q, keys, values, sinks, window, scale, new_assigned=True, extra=1.0):
    """got [pages, Hkv, 16] after one call against the plain form; q [B, T, Hq, D], keys[b] [L, Hkv, D]."""
    want = w0.astype(np.float64)
    touched = np.zeros(w0.shape[0::2], bool)
    tol = np.zeros(w0.shape)
    for b, L in enumerate(lens):
        L, nb = int(L), int(n[b])
        if L == 0 or nb == 0:
            continue
        _, mass, seen = pw.step(q[b], keys[b], values[b], L, nb, sinks, window, scale)
        c = np.arange(L)[seen]
        pg, sl = bt[b, c // 16], c % 16
        fresh = (c >= L - nb)[:, None] if new_assigned else np.zeros((len(c), 1), bool)
        want[pg, :, sl] = np.where(fresh, mass[seen], want[pg, :, sl] + mass[seen])
        rel = extra * pw.weights_tolerance(q[b, :nb], keys[b][seen], nb * q.shape[2] // keys[b].shape[1], L, scale)
        tol[pg, :, sl] += rel * mass[seen] + 2.0 ** -23 * want[pg, :, sl] + 1e-37
        touched[pg, sl] = True
    t = np.broadcast_to(touched[:, None, :], w0.shape)
    np.testing.assert_array_equal(got[~t].view(np.uint32), w0[~t].view(np.uint32))
    assert np.all(np.isfinite(got[t])), "non-finite weight"
    over = np.abs(got[t].astype(np.float64) - want[t]) / tol[t]
    assert over.size == 0 or over.max() <= 1, f"weight off by {over.max():.2f} of its bound"
    return want


def logical(c, L):
    return [bf16_to_f64(c.hist_k[b, :int(L[b])]) for b in range(c.B)], [bf16_to_f64(c.hist_v[b, :int(L[b])]) for b in range(c.B)]


def run_multi(m, window, seed=1, sinks=True, q_lens=True, one=False, fused=True, scale=None):
    """A several-token call (one: the one-token call) with weights, and without."""
    c, scale = m.c, m.c.scale if scale is None else scale
    kp, vp, bt = m.paged(seed, after=not fused)
    w0 = start_weights(kp.shape[0], c.Hkv, bt, m.base if fused else m.lens, seed)
    kd, vd, w = dev_bits(kp), dev_bits(vp), dev(w0)
    k2, v2 = dev_bits(kp), dev_bits(vp)
    q, kn, vn = dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new)
    if one:
        q, kn, vn = q[:, 0].contiguous(), kn[:, 0].contiguous(), vn[:, 0].contiguous()
    if not fused:
        kn = vn = None
    out, ref = (torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sk = dev(m.sinks) if sinks else None
    if one:
        da.decode_attn_paged_weights(q, kn, vn, kd, vd, w, dev(bt), dev(c.lens), sk, window, scale, out)
        da.decode_attn_paged(q, kn, vn, k2, v2, dev(bt), dev(c.lens), sk, window, scale, ref)
    else:
        ql = dev(m.n) if q_lens else None
        da.decode_attn_paged_multi_weights(q, kn, vn, kd, vd, w, dev(bt), dev(c.lens), sk, window, scale, out, q_lens=ql)
        da.decode_attn_paged_multi(q, kn, vn, k2, v2, dev(bt), dev(c.lens), sk, window, scale, ref, q_lens=ql)
    torch.cuda.synchronize()
    assert da.decode_attn_device_status() == 0
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    for a, b in ((kd, k2), (vd, v2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    keys, values = logical(c, c.lens)
    check_weights(w.cpu().numpy(), w0, bt, c.lens, m.n, bf16_to_f64(m.q), keys, values,
                  m.sinks.astype(np.float64) if sinks else None, window, scale, new_assigned=fused)
    return w.cpu().numpy()


EDGE = [1, 2, 15, 16, 17, 31, 33, 100, 257, 1000, 0]
HEADS = [(64, 8), (8, 8), (16, 1), (32, 4), (6, 3), (24, 12)]


def one_token(seed, Hq, Hkv, lens):
    return Multi(seed, Hq, Hkv, lens, [1 if L > 0 else 0 for L in lens], 1)


@pytest.mark.parametrize("Hq,Hkv", [h for h in HEADS if h != (6, 3)] + [(4, 2)])
@pytest.mark.parametrize("window", [0, 7, 100])
def test_one_token(Hq, Hkv, window):
    m = one_token(1000 + Hq + window, Hq, Hkv, EDGE)
    run_multi(m, window, seed=Hq, one=True)


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 1)])
def test_one_token_without_append_or_sinks(Hq, Hkv):
    """k_new None: token p is read from the cache and its weight is added like the others'."""
    m = one_token(1010 + Hq, Hq, Hkv, EDGE)
    run_multi(m, 0, one=True, fused=False)
    run_multi(m, 33, one=True, fused=False, sinks=False)
    run_multi(m, 0, one=True, sinks=False)


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 1), (1, 1)])
def test_one_long_sequence_over_the_whole_gpu(Hq, Hkv):
    m = one_token(1020 + Hq, Hq, Hkv, [20000, 3001])
    run_multi(m, 0, one=True)
    run_multi(m, 5003, one=True)


def test_many_slots_of_all_lengths():
    rng = np.random.default_rng(3)
    lens = [0 if rng.random() < 0.25 else int(rng.integers(1, 700)) for _ in range(200)]
    run_multi(one_token(1030, 16, 2, lens), 0, one=True)


def test_largest_batch():
    run_multi(one_token(1031, 2, 1, [1 + i % 40 for i in range(1024)]), 0, one=True)


def test_scores_far_apart():
    """Keys that grow along the sequence: probabilities from 1 down to underflow."""
    m = one_token(1040, 64, 8, [900, 300, 2000])
    ramp_keys(m, 12.0)
    run_multi(m, 0, one=True)
    run_multi(m, 0, one=True, scale=1.0)
    m = Multi(1041, 64, 8, [900, 300, 2000], [16, 16, 16], 16)
    ramp_keys(m, 12.0)
    run_multi(m, 0)


@pytest.mark.parametrize("Hq,Hkv", HEADS[:4] + [(4, 2)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 16, 33])
@pytest.mark.parametrize("window", [0, 7, 100])
def test_several_tokens(Hq, Hkv, T, window):
    """Up to 4 tokens and 32 rows per KV head: the decode kernel; below 64 rows the row-block
    kernel; from there tcgen05. The weights' own kernel takes all of them."""
    lens = [1, 4, 15, 16, 17, 33, 100, 257, 0]
    m = Multi(1100 + Hq + T + window, Hq, Hkv, lens, counts(T, lens, Hq + T + window), T)
    run_multi(m, window, seed=T + 1)


@pytest.mark.parametrize("T,lens", [(200, [1200, 200, 333, 17]), (700, [700, 701, 2000]), (130, [130, 5000])])
def test_prompt_chunks(T, lens):
    """Many query rows per KV head, whole prompts and chunks behind a history, windows that start
    inside a page and drop whole key blocks."""
    m = Multi(1200 + T, 16, 2, lens, [min(T, L) for L in lens], T)
    run_multi(m, 0)
    run_multi(m, 37)
    run_multi(m, 1000, q_lens=[L >= T for L in lens] and min(lens) < T)
    m = Multi(1201 + T, 16, 1, lens, [min(T, L) // 2 for L in lens], T)
    run_multi(m, 0, sinks=False)


def test_most_query_tokens_and_most_slots():
    """4096 new tokens of 16 query heads per KV head (65536 rows), and 1024 slots."""
    run_multi(Multi(1290, 16, 1, [4096, 100], [4096, 100], 4096), 0)
    lens = [1 + i % 40 for i in range(1024)]
    run_multi(Multi(1291, 2, 1, lens, [min(L, 3) for L in lens], 3), 0)
    run_multi(Multi(1292, 8, 1, lens, [min(L, 9) for L in lens], 9), 5)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (64, 8)])
@pytest.mark.parametrize("T", [4, 6, 16, 32])
def test_several_tokens_behind_a_long_history(Hq, Hkv, T):
    m = Multi(1300 + T + Hq, Hq, Hkv, [20000, 3000], [T, T - 1], T)
    run_multi(m, 0)


def test_windows_that_no_sequence_fills():
    """A window of the largest integer is no window."""
    for window in (1000, 1001, 2 ** 31 - 1):
        run_multi(one_token(1305, 16, 2, [1000, 17, 0, 300]), window, one=True)
        for T in (3, 9, 70):
            run_multi(Multi(1306 + T, 16, 2, [1000, 17, 0, 300], [T, min(T, 17), 0, T], T), window)


def test_counts_beyond_a_sequence_do_not_touch_it():
    m = Multi(1310, 8, 8, [10, 20], [2, 2], 2)
    kp, vp, bt = m.paged(1)
    w0 = start_weights(kp.shape[0], 8, bt, m.base, 1)
    w, out = dev(w0), torch.empty((2, 2, 8, 64), dtype=torch.bfloat16, device=DEV)
    da.decode_attn_paged_multi_weights(dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), dev_bits(kp), dev_bits(vp), w,
                                       dev(bt), dev(m.lens), None, 0, 0.125, out,
                                       q_lens=torch.tensor([3, 0], dtype=torch.int32, device=DEV))
    assert da.decode_attn_device_status() & da.DA_STATUS_BAD_SEQ_LEN
    np.testing.assert_array_equal(w.cpu().numpy().view(np.uint32), w0.view(np.uint32))


@pytest.mark.parametrize("one", [True, False])
def test_bad_pages_are_skipped(one):
    m = one_token(1320, 16, 2, [100, 60]) if one else Multi(1320, 16, 2, [100, 60], [9, 9], 9)
    kp, vp, bt = m.paged(1)
    w0 = start_weights(kp.shape[0], 2, bt, m.base, 1)
    bad = bt.copy()
    bad[0, 2], bad[1, 1] = -1, kp.shape[0]
    w = dev(w0)
    q, kn, vn = dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new)
    out = torch.empty_like(q)
    if one:
        da.decode_attn_paged_weights(q[:, 0].contiguous(), kn[:, 0].contiguous(), vn[:, 0].contiguous(), dev_bits(kp),
                                     dev_bits(vp), w, dev(bad), dev(m.lens), None, 0, 0.125, out[:, 0].contiguous())
    else:
        da.decode_attn_paged_multi_weights(q, kn, vn, dev_bits(kp), dev_bits(vp), w, dev(bad), dev(m.lens), None, 0, 0.125, out)
    assert da.decode_attn_device_status() & da.DA_STATUS_BAD_PAGE
    got = w.cpu().numpy()
    for b, pg in ((0, bt[0, 2]), (1, bt[1, 1])):
        np.testing.assert_array_equal(got[pg].view(np.uint32), w0[pg].view(np.uint32))
    assert np.all(got[bt[0, 0]] > w0[bt[0, 0]])


def test_lengths_beyond_the_bound_are_inactive():
    m = one_token(1330, 16, 2, [100, 60])
    kp, vp, bt = m.paged(1)
    w0 = start_weights(kp.shape[0], 2, bt, m.base, 1)
    w, q = dev(w0), dev_bits(m.q)[:, 0].contiguous()
    out = torch.full_like(q, float("nan"))
    kn = dev_bits(m.k_new)[:, 0].contiguous()
    da.decode_attn_paged_weights(q, kn, kn, dev_bits(kp), dev_bits(vp), w, dev(bt),
                                 torch.tensor([-3, 101], dtype=torch.int32, device=DEV), None, 0, 0.125, out, max_seq_len=100)
    assert da.decode_attn_device_status() & da.DA_STATUS_BAD_SEQ_LEN
    assert torch.all(out == 0)
    np.testing.assert_array_equal(w.cpu().numpy().view(np.uint32), w0.view(np.uint32))
    da.decode_attn_paged_weights(q, kn, kn, dev_bits(kp), dev_bits(vp), w, dev(bt),
                                 torch.zeros(2, dtype=torch.int32, device=DEV), None, 0, 0.125, out, max_seq_len=0)
    assert da.decode_attn_device_status() == 0 and torch.all(out == 0)


def test_sequences_that_share_their_first_pages():
    """Two sequences with a common prefix in the same pages: each adds its weights to the cells."""
    m = one_token(1340, 16, 2, [100, 70])
    m.c.hist_k[1, :48], m.c.hist_v[1, :48] = m.c.hist_k[0, :48], m.c.hist_v[0, :48]
    kp, vp, bt = m.paged(1)
    bt[1, :3] = bt[0, :3]
    w0 = start_weights(kp.shape[0], 2, bt, m.base, 1)
    w, q = dev(w0), dev_bits(m.q)[:, 0].contiguous()
    da.decode_attn_paged_weights(q, dev_bits(m.k_new)[:, 0].contiguous(), dev_bits(m.v_new)[:, 0].contiguous(),
                                 dev_bits(kp), dev_bits(vp), w, dev(bt), dev(m.lens), dev(m.sinks), 0, m.c.scale,
                                 torch.empty_like(q))
    keys, values = logical(m.c, m.c.lens)
    check_weights(w.cpu().numpy(), w0, bt, m.c.lens, m.n, bf16_to_f64(m.q), keys, values, m.sinks.astype(np.float64), 0,
                  m.c.scale)


# ---------------------------------------------------------------- fp8
def quantised(bits):
    """Codes (bytes) and scale of one row of bf16 bits: scale max |x| times the fp32 reciprocal of 448,
    codes the nearest e4m3 to x / scale."""
    x = torch.from_numpy(bf16_to_f64(bits).astype(np.float32))
    top = x.abs().max().numpy()
    scale = np.float32(top) * (np.float32(1) / np.float32(448)) if top > 0 else np.float32(1)
    return (x / torch.tensor(scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), scale


def append_fp8(blocks, c, bt):
    """The new token of every active sequence into copies of the 2176-byte blocks."""
    out = blocks.copy()
    for b, L in enumerate(c.lens):
        if L == 0:
            continue
        page, slot = bt[b, (L - 1) // 16], (L - 1) % 16
        for g in range(c.Hkv):
            (kc, ks), (vc, vs) = quantised(c.k_new[b, g]), quantised(c.v_new[b, g])
            blk = out[page, g]
            blk[slot * 64:slot * 64 + 64] = kc
            blk[1024 + slot:2048:16] = vc
            scales = blk[2048:].view(np.float32)
            scales[slot], scales[16 + slot] = ks, vs
    return out


def run_fp8(m, window, seed=1, fused=True, sinks=True):
    c = m.c
    held = m.base if fused else c.lens
    kp, vp, bt = paged_identity(c, held)
    kp, vp, bt = shuffle_pages(kp, vp, bt, seed, spare=4)
    cache = oracle.scatter_fp8(c.hist_k, c.hist_v, held, oracle.Fp8Cache.empty_paged(kp.shape[0], c.Hkv, 16, c.D), block_table=bt)
    start = np.ascontiguousarray(cache.blocks.reshape(kp.shape[0], c.Hkv, -1))
    blocks = append_fp8(start, c, bt) if fused else start
    w0 = start_weights(kp.shape[0], c.Hkv, bt, held, seed)
    kv, w = dev(start), dev(w0)
    q = dev_bits(m.q)[:, 0].contiguous()
    kn, vn = (dev_bits(c.k_new), dev_bits(c.v_new)) if fused else (None, None)
    out = torch.full_like(q, float("nan"))
    sk = dev(c.sinks) if sinks else None
    da.decode_attn_paged_fp8_weights(q, kn, vn, kv, w, dev(bt), dev(c.lens), sk, window, c.scale, out)
    torch.cuda.synchronize()
    assert da.decode_attn_device_status() == 0
    np.testing.assert_array_equal(kv.cpu().numpy(), blocks)
    if not fused:  # nothing is quantised: the output of the call without weights, bit for bit
        ref = torch.full_like(q, float("nan"))
        da.decode_attn_paged_fp8(q, None, None, kv, dev(bt), dev(c.lens), sk, window, c.scale, ref)
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    codes = torch.from_numpy(np.ascontiguousarray(blocks[..., :2048])).view(torch.float8_e4m3fn).double().numpy()
    scales = np.ascontiguousarray(blocks[..., 2048:]).view(np.float32).astype(np.float64)
    k = codes[..., :1024].reshape(-1, c.Hkv, 16, 64) * scales[..., :16, None]
    v = codes[..., 1024:].reshape(-1, c.Hkv, 64, 16).transpose(0, 1, 3, 2) * scales[..., 16:, None]
    keys, values = [], []
    for b, L in enumerate(c.lens):
        at = np.arange(L)
        keys.append(k[bt[b, at // 16], :, at % 16])
        values.append(v[bt[b, at // 16], :, at % 16])
    want = np.zeros(q.shape)
    for b, L in enumerate(c.lens):
        if L > 0:
            want[b] = pw.step(bf16_to_f64(m.q[b]), keys[b], values[b], int(L), 1, c.sinks.astype(np.float64) if sinks else None,
                              window, c.scale)[0][0]
    assert_close(out.double().cpu().numpy(), want, f"fp8 weights window={window}")
    # twice the bound: a score is (codes . q) * scale_k, one rounding more, and a query value below
    # fp16's normal range is off by up to 2^-25
    check_weights(w.cpu().numpy(), w0, bt, c.lens, m.n, bf16_to_f64(m.q), keys, values,
                  c.sinks.astype(np.float64) if sinks else None, window, c.scale, new_assigned=fused, extra=2.0)


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (8, 8), (16, 1), (32, 4), (4, 2)])
@pytest.mark.parametrize("window", [0, 7, 100])
def test_fp8(Hq, Hkv, window):
    run_fp8(one_token(1400 + Hq + window, Hq, Hkv, EDGE), window, seed=Hq)


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 1)])
def test_fp8_rows_as_torch_quantises_them(Hq, Hkv):
    """The appended bytes of rows whose largest values make the reciprocal and the division differ
    (and codes near a tie with them) are those of the torch expression on the GPU."""
    lens = [1 + i for i in range(128)]
    m = one_token(1420 + Hq, Hq, Hkv, lens)
    gen = np.random.default_rng(Hq)
    for b in range(128):  # every bf16 mantissa as a row's largest value
        for x in (m.c.k_new, m.c.v_new):
            x[b] = (gen.integers(0, 128, x[b].shape) | 0x3f00 | gen.integers(0, 2, x[b].shape) << 15).astype(np.uint16)
            x[b, :, 5] = 0x4000 | b
    kp, vp, bt = paged_identity(m.c, m.base)
    kv = torch.zeros((kp.shape[0], Hkv, 2176), dtype=torch.uint8, device=DEV)
    q, kn, vn = dev_bits(m.q)[:, 0].contiguous(), dev_bits(m.c.k_new), dev_bits(m.c.v_new)
    w = torch.zeros((kp.shape[0], Hkv, 16), device=DEV)
    da.decode_attn_paged_fp8_weights(q, kn, vn, kv, w, dev(bt), dev(m.c.lens), None, 0, m.c.scale, torch.empty_like(q))
    for x, at, scale_at in ((kn, None, 0), (vn, 1024, 16)):
        top = x.float().abs().amax(-1, keepdim=True)
        scale = top / 448
        codes = (x.float() / scale).to(torch.float8_e4m3fn).view(torch.uint8)
        for b in range(128):
            blk, slot = kv[int(bt[b, b // 16])], b % 16
            got = blk[:, slot * 64:slot * 64 + 64] if at is None else blk[:, at + slot:at + 1024:16]
            assert torch.equal(got, codes[b])
            assert torch.equal(blk[:, 2048:].contiguous().view(torch.float32)[:, scale_at + slot], scale[b, :, 0])


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 1)])
def test_fp8_long_and_without_append(Hq, Hkv):
    """The one long sequence at 8 KV heads has over 16384 tiles: the kernel of two CTAs per SM."""
    m = one_token(1410 + Hq, Hq, Hkv, [33000, 3001] if Hkv == 8 else [9000, 3001])
    run_fp8(m, 0)
    m = one_token(1411 + Hq, Hq, Hkv, EDGE)
    run_fp8(m, 0, fused=False)
    run_fp8(m, 50, fused=False, sinks=False)


# ---------------------------------------------------------------- levels, streams, graphs, determinism
@pytest.mark.parametrize("level", [1, 2])
def test_early_input_levels_do_not_change_the_weights(level):
    m, m4 = one_token(1500, 64, 8, [700, 20, 3000, 0, 64]), Multi(1501, 64, 8, [700, 20, 3000, 0, 64], [4, 2, 3, 0, 4], 4)
    a, a4 = run_multi(m, 0, one=True), run_multi(m4, 0)
    prev = da.decode_attn_set_early_inputs(level)
    try:
        b, b4 = run_multi(m, 0, one=True), run_multi(m4, 0)
    finally:
        da.decode_attn_set_early_inputs(prev)
    np.testing.assert_array_equal(a.view(np.uint32), b.view(np.uint32))
    np.testing.assert_array_equal(a4.view(np.uint32), b4.view(np.uint32))


def test_calls_behind_one_another_add_up():
    """Ten calls queued without a wait between them: each adds to the cells the one before wrote."""
    m = one_token(1510, 64, 8, [900, 33, 2500])
    kp, vp, bt = m.paged(1, after=True)
    w = dev(np.zeros((kp.shape[0], 8, 16), np.float32))
    q, kd, vd, btd, sl = dev_bits(m.q)[:, 0].contiguous(), dev_bits(kp), dev_bits(vp), dev(bt), dev(m.lens)
    out = torch.empty_like(q)
    for _ in range(10):
        da.decode_attn_paged_weights(q, None, None, kd, vd, w, btd, sl, None, 0, m.c.scale, out)
    one = dev(np.zeros((kp.shape[0], 8, 16), np.float32))
    da.decode_attn_paged_weights(q, None, None, kd, vd, one, btd, sl, None, 0, m.c.scale, out)
    total = torch.zeros_like(one)
    for _ in range(10):
        total += one
    assert torch.equal(w, total)


def test_two_streams_with_workspaces_of_their_own():
    jobs = [one_token(1520, 64, 8, [3000, 400]), one_token(1521, 64, 8, [250, 5000])]
    streams, args = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for m in jobs:
        kp, vp, bt = m.paged(1, after=True)
        args.append((m, dev_bits(m.q)[:, 0].contiguous(), dev_bits(kp), dev_bits(vp),
                     dev(np.zeros((kp.shape[0], 8, 16), np.float32)), dev(bt), dev(m.lens), bt))
    torch.cuda.synchronize()
    for s in streams:
        da.decode_attn_stream_reserve(s)
        da.decode_attn_weights_reserve(da.decode_attn_weights_workspace_bytes(2, 64, 8, 1, 5008), s)
    try:
        for _ in range(20):
            for s, (m, q, k, v, w, bt, sl, _) in zip(streams, args):
                with torch.cuda.stream(s):
                    da.decode_attn_paged_weights(q, None, None, k, v, w, bt, sl, None, 0, m.c.scale, torch.empty_like(q))
        torch.cuda.synchronize()
    finally:
        for s in streams:
            da.decode_attn_stream_release(s)
    for m, q, k, v, w, bt, sl, table in args:
        once = torch.zeros_like(w)
        da.decode_attn_paged_weights(q, None, None, k, v, once, bt, sl, None, 0, m.c.scale, torch.empty_like(q))
        total = torch.zeros_like(w)
        for _ in range(20):
            total += once
        assert torch.equal(w, total)


@pytest.mark.parametrize("T", [0, 3, 12])
def test_graph_survives_a_larger_call(T):
    """A captured call keeps its workspace when a later, larger call outgrows it; replayed after
    the lengths changed, it matches the eager call bit for bit."""
    def build(lens, seed):
        m = one_token(seed, 64, 8, lens) if T == 0 else Multi(seed, 64, 8, lens, [min(T, L) for L in lens], T)
        kp, vp, bt = m.paged(1)
        w0 = start_weights(kp.shape[0], 8, bt, m.base, 1)
        pick = (lambda x: x[:, 0].contiguous()) if T == 0 else (lambda x: x)
        return m, [pick(dev_bits(m.q)), pick(dev_bits(m.k_new)), pick(dev_bits(m.v_new)), dev_bits(kp), dev_bits(vp), dev(w0),
                   dev(bt), dev(m.lens), dev(m.sinks), 0, m.c.scale], dev(m.n)

    def launch(args, n, out):
        if T == 0:
            da.decode_attn_paged_weights(*args, out)
        else:
            da.decode_attn_paged_multi_weights(*args, out, q_lens=n)

    m, args, n = build([300, 40, 90], 1530 + T)
    out = torch.empty_like(args[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    da.decode_attn_stream_reserve(s)
    try:
        with torch.cuda.stream(s):
            launch(args, n, out)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                launch(args, n, out)
            big, big_args, big_n = build([5000, 300, 9000, 44, 700], 1540 + T)
            launch(big_args, big_n, torch.empty_like(big_args[0]))
            s.synchronize()
            args[7].copy_(torch.tensor([250, 37, 80], dtype=torch.int32))
            w0 = args[5].clone()
            eager, eager_out = list(args), torch.empty_like(out)
            eager[3], eager[4], eager[5] = args[3].clone(), args[4].clone(), w0.clone()
            g.replay()
            launch(eager, n, eager_out)
            s.synchronize()
        assert da.decode_attn_device_status(s) == 0
        assert torch.equal(out.view(torch.int16), eager_out.view(torch.int16))
        assert torch.equal(args[5].view(torch.int32), eager[5].view(torch.int32))
        del g
    finally:
        da.decode_attn_stream_release(s)


def test_capture_without_a_workspace_is_refused():
    m = one_token(1550, 64, 8, [300, 40])
    kp, vp, bt = m.paged(1)
    w = dev(start_weights(kp.shape[0], 8, bt, m.base, 1))
    args = [dev_bits(m.q)[:, 0].contiguous(), dev_bits(m.k_new)[:, 0].contiguous(), dev_bits(m.v_new)[:, 0].contiguous(),
            dev_bits(kp), dev_bits(vp), w, dev(bt), dev(m.lens), None, 0, 0.125]
    out = torch.empty_like(args[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    da.decode_attn_stream_reserve(s)
    try:
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with pytest.raises(da.DecodeAttnError) as e:
                with torch.cuda.graph(g, stream=s):
                    da.decode_attn_paged_weights(*args, out)
            assert e.value.code == -3
    finally:
        da.decode_attn_stream_release(s)


def test_refusals():
    m = one_token(1560, 16, 2, [100, 60])
    kp, vp, bt = m.paged(1)
    w = dev(start_weights(kp.shape[0], 2, bt, m.base, 1))
    q, kn, k = dev_bits(m.q)[:, 0].contiguous(), dev_bits(m.k_new)[:, 0].contiguous(), dev_bits(kp)
    out, btd, sl = torch.empty_like(q), dev(bt), dev(m.lens)

    def call(**kw):
        a = dict(q=q, k_new=kn, v_new=kn, k_cache=k, v_cache=k, weights=w, block_table=btd, seq_lens=sl, sinks=None, window=0,
                 scale=0.125, out=out)
        a.update(kw)
        da.decode_attn_paged_weights(**a)

    for name, bad in (("q", q.float()), ("q", q.transpose(0, 1)), ("k_new", kn[:1]), ("weights", w.double()),
                      ("weights", w[:, :, :8]), ("block_table", btd.long()), ("seq_lens", sl[:1]), ("out", out.cpu()),
                      ("v_cache", k[:, :, :, ::2]), ("sinks", torch.zeros(3, device=DEV))):
        with pytest.raises(ValueError, match=name):
            call(**{name: bad})
    with pytest.raises(ValueError):
        call(v_new=None)
    for kw in (dict(scale=-1.0), dict(window=-1), dict(max_seq_len=10 ** 6)):
        with pytest.raises(da.DecodeAttnError) as e:
            call(**kw)
        assert e.value.code == -1
