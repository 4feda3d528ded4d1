"""GPU parity of qk_norm_rope against the definition in fp64: with norms within bf16's half step 2^-8 of
the value plus 2^-20 of the larger of the pair (fp32 products, sums of 64 squares, one division and root:
fewer than 16 roundings of 2^-24 each), without norms bit for bit (fp32 products and sums rounded one by one); values copied bit for bit."""
import numpy as np
import pytest
import torch

import paged_decode_attention_kv_gb300 as da

pytestmark = pytest.mark.gpu
DEV = "cuda"


def tables(n, base=10000.0):
    a = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(32, dtype=torch.float64) / 32)
    return a.cos().float().to(DEV), a.sin().float().to(DEV)


def axis_of(sections, interleaved):
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while len(out) < 32:
        for a in range(len(left)):
            if left[a] > 0:
                left[a] -= 1
                out.append(a)
    return out


def plain(x, pos, cos, sin, w, eps, axis):
    """fp64; x [N, H, 64], pos [axes, N]."""
    y = x.double()
    if w is not None:
        y = y / ((y * y).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    at = pos.long()[torch.tensor(axis, device=DEV)].T
    i = torch.arange(32, device=DEV)
    c, s = cos.double()[at, i][:, None], sin.double()[at, i][:, None]
    a, b = y[..., :32], y[..., 32:]
    return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([torch.maximum(a.abs(), b.abs())] * 2, -1)


def fp32_rotation(x, pos, cos, sin, axis):
    at = pos.long()[torch.tensor(axis, device=DEV)].T
    i = torch.arange(32, device=DEV)
    c, s = cos[at, i][:, None], sin[at, i][:, None]
    a, b = x.float()[..., :32], x.float()[..., 32:]
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    return torch.cat([ac - bs, bc + as_], -1).to(torch.bfloat16)


def packed(N, Hq, Hkv, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((N, Hq + 2 * Hkv, 64), generator=g, device=DEV).to(torch.bfloat16)
    w = [0.5 + torch.rand(64, generator=g, device=DEV) for _ in range(2)]
    return x, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w, g


def check(got, want, size):
    err = (got.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all(), float((err - 2.0 ** -8 * want.abs()).max())


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (1, 1), (7, 3), (12, 1)])
@pytest.mark.parametrize("N", [1, 2, 65, 1000])
@pytest.mark.parametrize("sections,interleaved", [(None, False), ((16, 8, 8), False), ((12, 10, 10), True), ((5, 27), False), ((32, 0, 0), False)])
def test_matches_definition(Hq, Hkv, N, sections, interleaved):
    x, q, k, v, (wq, wk), g = packed(N, Hq, Hkv, N + Hq)
    cos, sin = tables(4096)
    axes = 1 if sections is None else len(sections)
    pos = torch.randint(0, 4096, (axes, N), generator=g, device=DEV, dtype=torch.int32)
    axis = [0] * 32 if sections is None else axis_of(sections, interleaved)
    keep = x.clone()
    for norm in (True, False):
        qo, ko, vo = (torch.full(y.shape, float("nan"), dtype=torch.bfloat16, device=DEV) for y in (q, k, v))
        da.qk_norm_rope(q, k, pos if axes > 1 else pos[0], cos, sin, qo, ko, q_weight=wq if norm else None, k_weight=wk if norm else None,
                        sections=sections, interleaved=interleaved, v=v, v_out=vo)
        assert da.decode_attn_device_status() == 0
        assert torch.equal(vo, v) and torch.equal(x, keep)
        for y, got, w in ((q, qo, wq), (k, ko, wk)):
            if norm:
                check(got, *plain(y, pos, cos, sin, w, 1e-6, axis))
            else:
                assert torch.equal(got, fp32_rotation(y, pos, cos, sin, axis))


def test_in_place_without_values_and_one_norm():
    """In place in the packed rows; the value rows, and a norm of the keys alone."""
    x, q, k, v, (wq, wk), g = packed(33, 8, 2, 5)
    cos, sin = tables(100)
    pos = torch.arange(33, device=DEV, dtype=torch.int32)
    want = [plain(q, pos[None], cos, sin, None, 0, [0] * 32), plain(k, pos[None], cos, sin, wk, 1e-5, [0] * 32)]
    keep = v.clone()
    da.qk_norm_rope(q, k, pos, cos, sin, q, k, k_weight=wk, eps=1e-5)
    check(q, *want[0])
    check(k, *want[1])
    assert torch.equal(v, keep)


def test_rows_of_zeros_infinities_and_nan_stay_their_own():
    """A row of zeros stays zeros; a row with an infinity or a NaN spoils no other row."""
    x, q, k, v, (wq, wk), g = packed(4, 8, 8, 6)
    q[1, 2] = 0
    q[1, 3, 5] = float("inf")
    k[2, 7, 0] = float("nan")
    cos, sin = tables(8)
    pos = torch.tensor([0, 3, 7, 1], device=DEV, dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    da.qk_norm_rope(q, k, pos, cos, sin, qo, ko, q_weight=wq, k_weight=wk)
    assert not qo[1, 2].any()
    bad_q = ~qo.isfinite().all(-1)
    bad_k = ~ko.isfinite().all(-1)
    assert bad_q.nonzero().tolist() == [[1, 3]] and bad_k.nonzero().tolist() == [[2, 7]]


def test_shapes_of_a_batch_and_of_multi_token_rows():
    """[B, T, heads, 64] views of packed rows, a row stride above the heads, one token."""
    x, *_ , g = packed(12, 8, 2, 7)
    big = torch.zeros((3, 4, 20, 64), dtype=torch.bfloat16, device=DEV)
    big[:, :, :12] = x.view(3, 4, 12, 64)
    cos, sin = tables(64)
    pos = torch.randint(0, 64, (3, 4), generator=g, device=DEV, dtype=torch.int32)
    out = [torch.empty((3, 4, h, 64), dtype=torch.bfloat16, device=DEV) for h in (8, 2)]
    flat = [torch.empty((12, h, 64), dtype=torch.bfloat16, device=DEV) for h in (8, 2)]
    da.qk_norm_rope(big[:, :, :8], big[:, :, 8:10], pos, cos, sin, *out)
    da.qk_norm_rope(x[:, :8], x[:, 8:10], pos.view(-1), cos, sin, *flat)
    for a, b in zip(out, flat):
        assert torch.equal(a.view(b.shape), b)


def test_positions_outside_the_tables():
    x, q, k, v, w, g = packed(3, 4, 1, 8)
    cos, sin = tables(10)
    out = [torch.empty_like(q), torch.empty_like(k)]
    da.qk_norm_rope(q, k, torch.tensor([2, 10, -1], device=DEV, dtype=torch.int32), cos, sin, *out)
    assert da.decode_attn_device_status() == da.DA_STATUS_BAD_POSITION
    assert torch.equal(out[0], fp32_rotation(q, torch.tensor([[2, 0, 0]], device=DEV), cos, sin, [0] * 32))


def test_the_bits_of_the_fused_rotation():
    """Without a norm: what decode_attn_paged_rope appends."""
    B, L, H = 3, 20, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    q, k, v = (torch.randn((B, h, 64), generator=g, device=DEV).to(torch.bfloat16) for h in (8, H, H))
    cos, sin = tables(64)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    table = torch.arange(2 * B, dtype=torch.int32, device=DEV).view(B, 2)
    pools = [torch.zeros((2 * B, H, 16, 64), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    out = [torch.empty_like(q) for _ in range(2)]
    da.decode_attn_paged_rope(q, k, v, pools[0], pools[1], table, lens, None, cos, sin, 0, 0.125, out[0])
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    da.qk_norm_rope(q, k, lens - 1, cos, sin, qr, kr)
    da.decode_attn_paged(qr, kr, v, pools[2], pools[3], table, lens, None, 0, 0.125, out[1])
    assert torch.equal(pools[0], pools[2]) and torch.equal(out[0], out[1])
