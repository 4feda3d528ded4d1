"""A step whose chunk has no token, in a batch of sequences: rotation, append and attention all return, and nothing changes."""
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from test_gpu_qk_norm_rope import DEV, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [False, True])
def test_no_token(counts):
    def rows(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    cos, sin = tables(16)
    kv = torch.randint(0, 120, (8, 2, da.FP8_BLOCK_BYTES), dtype=torch.uint8, device=DEV)
    before = kv.clone()
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    lens = torch.tensor([9, 0], dtype=torch.int32, device=DEV)
    n = torch.zeros(2, dtype=torch.int32, device=DEV) if counts else None
    x = rows(2, 0, 12, 64)
    q, k, v, out = rows(2, 0, 8, 64), rows(2, 0, 2, 64), rows(2, 0, 2, 64), rows(2, 0, 8, 64)
    for pos, sections in ((torch.empty((2, 0), dtype=torch.int32, device=DEV), None), (torch.empty((3, 0), dtype=torch.int32, device=DEV), (12, 10, 10))):
        da.qk_norm_rope(x[:, :, :8], x[:, :, 8:10], pos, cos, sin, q, k, sections=sections, v=x[:, :, 10:], v_out=v)
    da.kv_append_fp8(k, v, kv, lens, block_table=table, q_lens=n)
    da.kv_append_fp8(k, v, kv[:2].view(2, 2, 1, da.FP8_BLOCK_BYTES), lens, q_lens=n)
    assert da.decode_attn_paged_fp8_multi(q, k, v, kv, table, lens, None, 0, 0.125, out, q_lens=n) is out
    torch.cuda.synchronize()
    assert da.decode_attn_device_status() == 0 and torch.equal(kv, before)


def test_a_wrong_tensor_is_still_named():
    kv = torch.zeros((8, 2, da.FP8_BLOCK_BYTES), dtype=torch.uint8, device=DEV)
    lens, table = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    k = torch.empty((2, 0, 2, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="v_new"):
        da.kv_append_fp8(k, k.float(), kv, lens, block_table=table)
    with pytest.raises(ValueError, match="v_new"):
        da.decode_attn_paged_fp8_multi(torch.empty((2, 0, 8, 64), dtype=torch.bfloat16, device=DEV), k, k[..., :32], kv, table, lens, None, 0, 0.125,
                                       torch.empty((2, 0, 8, 64), dtype=torch.bfloat16, device=DEV))
