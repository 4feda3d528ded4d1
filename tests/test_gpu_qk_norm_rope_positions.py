"""The shapes that the positions of qk_norm_rope come in: the rows' own leading dimensions, with an axis ahead of them
or none, or all tokens in one. The same positions give the same bits."""
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from test_gpu_qk_norm_rope import DEV, packed, tables

pytestmark = pytest.mark.gpu


def rotate(x, pos, cos, sin, **kw):
    q, k = x[..., :8, :], x[..., 8:10, :]
    out = [torch.empty(y.shape, dtype=torch.bfloat16, device=DEV) for y in (q, k)]
    da.qk_norm_rope(q, k, pos, cos, sin, *out, **kw)
    return torch.cat([y.reshape(-1, y.shape[-2] * 64) for y in out], 1)


@pytest.mark.parametrize("sections", [(32,), (12, 20), (12, 10, 10)])
@pytest.mark.parametrize("shape", [(3, 4), (2, 2, 3), (1, 12), (12, 1)])
def test_positions_of_rows_in_batches(sections, shape):
    x, *_, g = packed(12, 8, 2, 11)
    cos, sin = tables(64)
    axes = len(sections)
    pos = torch.randint(0, 64, (axes, 12), generator=g, device=DEV, dtype=torch.int32)
    want = rotate(x, pos, cos, sin, sections=sections)
    rows = x.view(*shape, 12, 64)
    assert torch.equal(rotate(rows, pos, cos, sin, sections=sections), want)
    assert torch.equal(rotate(rows, pos.view(axes, *shape), cos, sin, sections=sections), want)
    if axes == 1:  # one axis needs no dimension of its own
        for p in (pos[0], pos[0].view(shape)):
            assert torch.equal(rotate(rows, p, cos, sin, sections=sections), want)
            assert torch.equal(rotate(rows, p, cos, sin), want)


def test_positions_of_another_count_are_refused():
    x, *_ = packed(12, 8, 2, 12)
    cos, sin = tables(64)
    rows = x.view(3, 4, 12, 64)
    for shape in ((2, 12), (3, 11), (3, 4, 3), (12,), (3, 4)):
        with pytest.raises(ValueError, match="positions"):
            rotate(rows, torch.zeros(shape, dtype=torch.int32, device=DEV), cos, sin, sections=(12, 10, 10))
    for shape in ((11,), (4, 3), (2, 12)):
        with pytest.raises(ValueError, match="positions"):
            rotate(rows, torch.zeros(shape, dtype=torch.int32, device=DEV), cos, sin, sections=(32,))
    with pytest.raises(ValueError, match="sections"):
        rotate(rows, torch.zeros((0, 12), dtype=torch.int32, device=DEV), cos, sin, sections=())
