"""GPU: what a call leaves in the weights workspace does not reach the next call's weights. Rows whose
scores are all -inf (and no sink) have no denominator: they are written as zeros, and their weights
are zero whatever the workspace held."""
import numpy as np
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from test_gpu_decode import dev, dev_bits
from test_gpu_weights import start_weights
from test_oracle_multi import Multi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,lens", [(0, [100, 33]), (2, [100, 33]), (5, [100, 33]), (5, [9000, 33]), (16, [100, 33]),
                                    (16, [9000, 33]), (64, [200, 64])])
def test_rows_of_infinite_scores_take_no_weight(T, lens):
    n = max(T, 1)
    m = Multi(2060 + T, 64, 8, lens, [n] * len(lens), n)
    m.c.hist_k[..., 0] = 0xff80                          # -inf
    m.k_new[..., 0] = 0xff80
    m.q[..., 0] = 0x3f80                                 # 1
    kp, vp, bt = m.paged(1)
    w0 = start_weights(kp.shape[0], 8, bt, m.base, 1)
    pick = (lambda x: x) if T else (lambda x: x[:, 0].contiguous())
    q, kn, vn, btd, sl = pick(dev_bits(m.q)), pick(dev_bits(m.k_new)), pick(dev_bits(m.v_new)), dev(bt), dev(m.lens)
    call = da.decode_attn_paged_multi_weights if T else da.decode_attn_paged_weights
    # a call before it with finite scores but for the first token's, which is NaN: so are its denominators
    k0, kn0 = dev_bits(kp), kn.clone()
    k0[..., 0] = kn0[..., 0] = 0
    for b in range(len(lens)):
        if lens[b] > n:
            k0[int(bt[b, 0]), :, 0] = float("nan")
        else:
            kn0[b, 0] = float("nan")
    w = dev(w0)
    scratch = w.clone()
    call(q, kn0, vn, k0, dev_bits(vp), scratch, btd, sl, None, 0, m.c.scale, torch.empty_like(q))
    assert bool(scratch[int(bt[0, 0])].isnan().all())
    call(q, kn, vn, dev_bits(kp), dev_bits(vp), w, btd, sl, None, 0, m.c.scale, torch.empty_like(q))
    assert da.decode_attn_device_status() == 0
    want = w0.copy()
    for b, L in enumerate(m.lens):
        j = np.arange(L - n, L)
        want[bt[b, j // 16], :, j % 16] = 0
    np.testing.assert_array_equal(w.cpu().numpy().view(np.uint32), want.view(np.uint32))
