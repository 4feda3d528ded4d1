"""What a step of new tokens over an fp8 cache meets at its edges: infinities and NaN in one sequence of a batch, a whole
step captured into a graph and replayed on other inputs, the largest batch."""
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from test_gpu_qk_norm_rope import DEV, tables

pytestmark = pytest.mark.gpu


def rows(*shape, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def ints(*shape, lo=0, hi=64, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("T", [4, 16, 150])
@pytest.mark.parametrize("what", ["new key", "new value", "cached scales", "cached codes"])
def test_nan_stays_in_its_sequence(T, what):
    """Segments of several sequences follow one another in a CTA: the other sequences' outputs keep their bits."""
    lens = torch.tensor([T + 100, T + 37, T + 500, T + 1, T + 64], device=DEV, dtype=torch.int32)
    B, w = 5, (T + 500 + 15) // 16
    q, k, v = rows(B, T, 64, 64, seed=1), rows(B, T, 8, 64, seed=2), rows(B, T, 8, 64, seed=3)
    table = torch.arange(B * w, device=DEV, dtype=torch.int32).view(B, w)
    hist = [rows(B, w * 16, 8, 64, seed=s) for s in (4, 5)]
    before = lens - T
    outs = []
    for bad in (False, True):
        kv = torch.zeros((B * w, 8, da.FP8_BLOCK_BYTES), dtype=torch.uint8, device=DEV)
        da.kv_append_fp8(*hist, kv, before, block_table=table, q_lens=before)
        kb, vb = k.clone(), v.clone()
        if bad and what == "new key":
            kb[2, T // 2, :, 5] = float("nan")
        if bad and what == "new value":
            vb[2, T // 2, :, 5] = float("inf")
        if bad and what == "cached scales":
            kv.view(torch.float32)[int(table[2, 3]), :, 512:544] = float("inf")
        if bad and what == "cached codes":
            kv[int(table[2, 3])] = 0xFF
        out = torch.empty_like(q)
        da.decode_attn_paged_fp8_multi(q, kb, vb, kv, table, lens, None, 0, 0.125, out)
        assert da.decode_attn_device_status() == 0
        outs.append(out)
    others = [0, 1, 3, 4]
    assert torch.equal(outs[0][others], outs[1][others]) and outs[0].isfinite().all()
    assert not outs[1][2, -1].isfinite().all()


def test_a_captured_step():
    B, T, w = 3, 6, 8
    x, pos = rows(B * T, 80, 64, seed=1), ints(3, B * T)
    lens = torch.tensor([40, 6, 100], device=DEV, dtype=torch.int32)
    sinks, wq = rows(64, seed=2).float(), 0.5 + rows(64, seed=3).float().abs()
    table = torch.arange(B * w, device=DEV, dtype=torch.int32).view(B, w)
    kv = torch.zeros((B * w, 8, da.FP8_BLOCK_BYTES), dtype=torch.uint8, device=DEV)
    cos, sin = tables(64)
    q, k, v = (torch.empty((B, T, h, 64), dtype=torch.bfloat16, device=DEV) for h in (64, 8, 8))
    out, back = torch.empty_like(q), [torch.zeros((B, 100, 8, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def step():
        da.qk_norm_rope(x[:, :64], x[:, 64:72], pos, cos, sin, q.view(-1, 64, 64), k.view(-1, 8, 64), q_weight=wq, k_weight=wq,
                        sections=(12, 10, 10), interleaved=True, v=x[:, 72:], v_out=v.view(-1, 8, 64))
        da.decode_attn_paged_fp8_multi(q, k, v, kv, table, lens, sinks, 0, 0.125, out)
        da.kv_read_fp8(kv, lens, *back, block_table=table)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for seed in (11, 12):
        x.copy_(rows(B * T, 80, 64, seed=seed))
        lens.copy_(torch.tensor([40 + seed, 6, 100 - seed]))
        got = []
        for run in (graph.replay, step):
            for t in (kv, out, *back):
                t.zero_()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            got.append([t.clone() for t in (kv, out, *back)])
        assert all(torch.equal(a, b) for a, b in zip(*got))
    assert da.decode_attn_device_status() == 0


def test_the_largest_batch():
    """1024 sequences at once, and 64 at a time: the sums in another order, each output rounded to bf16."""
    B, T, w = 1024, 5, 4
    lens, table = ints(B, lo=T, hi=60, seed=5), torch.randperm(B * w, device=DEV).int().view(B, w)
    q, k, v = rows(B, T, 64, 64, seed=1), rows(B, T, 8, 64, seed=2), rows(B, T, 8, 64, seed=3)
    kv = torch.zeros((B * w, 8, da.FP8_BLOCK_BYTES), dtype=torch.uint8, device=DEV)
    out, parts = torch.empty_like(q), torch.empty_like(q)
    da.decode_attn_paged_fp8_multi(q, k, v, kv, table, lens, None, 0, 0.125, out)
    for i in range(0, B, 64):
        at = slice(i, i + 64)
        da.decode_attn_paged_fp8_multi(q[at], k[at], v[at], kv, table[at], lens[at], None, 0, 0.125, parts[at])
    assert da.decode_attn_device_status() == 0
    a, b = out.float(), parts.float()
    assert ((a - b).abs() <= 2 * 2.0 ** -8 * a.abs() + 2e-3).all()
