"""CPU: how the binding reads the tokens of a view: their count, and the elements from one to the next."""
import pytest
import torch

import paged_decode_attention_kv_gb300 as da


def rows(x, heads):
    return da._token_rows("x", x, heads, -1)  # (-1: what a tensor on the CPU has for a device)


def test_views():
    x = torch.zeros(3, 4, 12 * 64, dtype=torch.bfloat16)
    assert rows(x.view(12, 12, 64)[:, 8:10], 2) == (12, 768)
    assert rows(x.view(3, 4, 12, 64)[:, :, :8], 8) == (12, 768)
    assert rows(x.view(3, 4, 12, 64)[:, 1:2, :8], 8) == (3, 4 * 768)
    assert rows(x.view(3, 4, 12, 64)[1:2, 1:2, :8], 8) == (1, 512)
    assert rows(x.view(3, 4, 12, 64)[:0], 12) == (0, 768)
    assert rows(x.view(3, 4, 12, 64)[:, :0], 12) == (0, 768)


def test_one_token_of_rows_of_odd_width():
    """The distance to the next token does not matter where there is none (the library takes multiples of 8 elements)."""
    x = torch.zeros(5, 12 * 64 + 3, dtype=torch.bfloat16)
    one = x[:, :768].unflatten(1, (12, 64))[:1]
    assert one.stride(0) % 8 != 0
    assert rows(one, 12) == (1, 768)
    assert rows(one[:, :8], 8) == (1, 512)


def test_tokens_that_are_not_evenly_spaced(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(3, 4, 12, 64, dtype=torch.bfloat16)
    for bad in (x[:, :3], x[:, :, :, :32], x.transpose(0, 1), x.float()):
        with pytest.raises(ValueError, match="evenly spaced"):
            rows(bad, 12)
