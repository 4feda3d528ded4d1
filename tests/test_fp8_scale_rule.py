"""CPU checks of the fp8 scale rules: the argument checks of decode_attn_paged_fp8_weights_rule, and how
far the two rules are apart."""
import numpy as np
import pytest

import paged_decode_attention_kv_gb300 as da
from test_abi import P, _shape


@pytest.fixture(scope="module")
def lib():
    from paged_decode_attention_kv_gb300 import build
    build.build()
    return da.load_library()


def call(lib, rule, s):
    return lib.decode_attn_paged_fp8_weights_rule(P, P, P, P, P, P, P, None, 0, 0.125, rule, P, s, 16, 16, 64, 200, None)


def test_rules_and_others(lib):
    for rule in (da.DA_FP8_SCALE_RECIPROCAL, da.DA_FP8_SCALE_DIVIDE):
        assert call(lib, rule, _shape(B=0)) == 0
    for rule in (-1, 2, 448):
        assert call(lib, rule, _shape(B=0)) == -1
        assert call(lib, rule, _shape()) == -1


def test_rules_differ_by_one_unit_in_the_last_place():
    top = ((0x4000 | np.arange(128, dtype=np.uint32)) << 16).view(np.float32)  # every bf16 mantissa
    divide, reciprocal = top / np.float32(448), top * (np.float32(1) / np.float32(448))
    apart = np.abs(divide.view(np.int32) - reciprocal.view(np.int32))
    assert apart.max() == 1 and apart.sum() == 71
