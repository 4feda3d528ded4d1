"""The bounded-wait failure paths of decode_attn_paged_fp8_multi, driven without a real stall: one warp of each role of
the tcgen05 kernel gives up at a wait that is over, early and in mid-stream, and so does the decode kernel's first worker.
The call reports DA_STATUS_TIMEOUT, and the next two, whose segments are shared between CTAs (so that
arrival counters left behind would show), match the oracle with a clean status."""
import pytest
import torch

import oracle
import paged_decode_attention_kv_gb300 as da
from test_gpu_decode import DEV, assert_close, dev, dev_bits
from test_gpu_fp8 import to_dev
from test_oracle_multi import Multi
from test_oracle_multi_fp8 import fp8_paged

pytestmark = pytest.mark.gpu
ROWS, OPERANDS, COPIES, PRODUCTS, QUERIES = range(5)


class Step:
    def __init__(self, seed, lens, T, Hkv=2):
        self.m = m = Multi(seed, 8 * Hkv, Hkv, lens, [min(L, T) for L in lens], T)
        blocks, bt, _ = fp8_paged(m, 1)
        self.args = [dev_bits(m.q), dev_bits(m.k_new), dev_bits(m.v_new), to_dev(blocks), dev(bt), dev(m.lens), dev(m.sinks), 0, m.c.scale]
        self.n = dev(m.n)
        self.want = oracle.decode_multi_fp8(m.q, m.k_new, m.v_new, blocks, m.lens, m.sinks, 0, m.c.scale, block_table=bt, q_lens=m.n)

    def call(self):
        out = torch.empty((self.m.c.B, self.m.T, self.m.c.Hq, 64), dtype=torch.bfloat16, device=DEV)
        da.decode_attn_paged_fp8_multi(*self.args, out, q_lens=self.n)
        return out, da.decode_attn_device_status()

    def check_expiry(self, tile):
        da.decode_attn_test_expire_wait(tile)
        _, status = self.call()
        assert status == da.DA_STATUS_TIMEOUT
        for _ in range(2):
            out, status = self.call()
            assert status == 0
            assert_close(out.double().cpu().numpy(), self.want, f"after an expired wait at {tile}")


@pytest.fixture(scope="module")
def folded():
    """Few long segments: their partials are folded by a kernel of its own."""
    return Step(3100, [9000, 700, 40], 16)


@pytest.fixture(scope="module")
def counted():
    """More segments than a quarter of the CTAs: the last of the CTAs that share one folds its partials."""
    return Step(3110, [300 + 31 * b % 900 for b in range(60)], 16)


@pytest.fixture(scope="module")
def short():
    """Three to four segments of one unit per CTA."""
    return Step(3115, [17 + 7 * b % 47 for b in range(300)], 16, Hkv=4)


@pytest.mark.parametrize("role", [ROWS, OPERANDS, COPIES, PRODUCTS, QUERIES])
def test_the_first_wait(folded, role):
    folded.check_expiry(role)


@pytest.mark.parametrize("role,i", [(OPERANDS, 1), (OPERANDS, 2), (COPIES, 1), (COPIES, 3)])
def test_in_mid_stream(counted, role, i):
    counted.check_expiry(8 * i + role)


@pytest.mark.parametrize("role,i", [(ROWS, 1), (ROWS, 2), (PRODUCTS, 1), (PRODUCTS, 2), (QUERIES, 1), (QUERIES, 2)])
def test_between_segments(short, role, i):
    short.check_expiry(8 * i + role)


@pytest.mark.parametrize("tile", [0, 2])
def test_up_to_four_tokens(tile):
    Step(3120, [20000, 500], 4).check_expiry(tile)


def test_an_expiry_that_no_wait_meets():
    step = Step(3130, [50], 16)
    da.decode_attn_test_expire_wait(8 * 1000)
    for _ in range(2):
        out, status = step.call()
        assert status == 0
        assert_close(out.double().cpu().numpy(), step.want)
