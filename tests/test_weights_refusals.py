"""CPU: what the calls with weights cannot do they refuse before anything is launched (a refusal after
the attention would leave the new tokens appended and their weights unwritten)."""
import pytest

import paged_decode_attention_kv_gb300 as da
from test_abi import _shape
from test_weights_plain import call


@pytest.fixture(scope="module")
def lib():
    from paged_decode_attention_kv_gb300 import build
    build.build()
    return da.load_library()


def test_more_key_blocks_than_a_grid_holds(lib):
    """512 query rows, 512 (sequence, KV head) pairs, 2^31 - 1 positions: 2^32 blocks of 256 keys. Refused
    as a shape, ahead of the first CUDA call (which fails here, without a device)."""
    wide = dict(s=_shape(B=64, Hq=64, Hkv=8), T=64, maxp=2 ** 27, maxlen=2 ** 31 - 1)
    assert call(lib, "multi", **wide) == -2
    assert call(lib, "multi", window=2 ** 30, **wide) == -2


def test_a_query_of_one_dimension_is_named(monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(da, "_paged_tensors", lambda *a: (0, 0, 0, 0, 0, 2, 1, 4, 8))
    q = torch.zeros(1024, dtype=torch.bfloat16)
    for one in (da.decode_attn_paged_weights, lambda q, *a: da.decode_attn_paged_fp8_weights(q, *a[:3], *a[4:])):
        with pytest.raises(ValueError, match="q must be"):
            one(q, None, None, None, None, None, None, None, None, 0, 0.125, q)
