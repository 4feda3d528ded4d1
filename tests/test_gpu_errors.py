"""GPU: a workspace that cannot be allocated is an error of its own call alone; the calls after it run."""
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from test_gpu_decode import dev, dev_bits
from test_gpu_weights import one_token

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reserve", [da.decode_attn_weights_reserve, da.decode_attn_multi_reserve, da.decode_attn_reserve])
def test_calls_after_a_refused_reservation(reserve):
    m = one_token(6000, 64, 8, [300, 40])
    kp, vp, bt = m.paged(1, after=True)
    q, k, v, btd, sl = dev_bits(m.q)[:, 0].contiguous(), dev_bits(kp), dev_bits(vp), dev(bt), dev(m.lens)
    w = torch.zeros(k.shape[:3], device="cuda")

    def run():
        outs = [torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)[:, None]]
        weights, nl, kept = w.clone(), torch.zeros_like(sl), torch.zeros((2, 8, 32), dtype=torch.int32, device="cuda")
        kc, vc = k.clone(), v.clone()
        da.decode_attn_paged(q, None, None, kc, vc, btd, sl, None, 0, 0.125, outs[0])
        da.decode_attn_paged_weights(q, None, None, kc, vc, weights, btd, sl, None, 0, 0.125, outs[1])
        da.decode_attn_paged_multi(q[:, None], k.new_zeros((2, 1, 8, 64)), k.new_zeros((2, 1, 8, 64)), kc, vc, btd, sl, None, 0, 0.125,
                                   outs[2])
        da.kv_evict(kc, vc, weights, btd, sl, nl, kept, 2, 8)
        torch.cuda.synchronize()
        return outs + [weights, nl, kept, kc, vc]

    want = run()
    with pytest.raises(da.DecodeAttnError) as e:
        reserve(1 << 44)                       # 16 TiB
    assert e.value.code == -4 and "memory" in str(e.value)
    for a, b in zip(run(), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert da.decode_attn_device_status() == 0
