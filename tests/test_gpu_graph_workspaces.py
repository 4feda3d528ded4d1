"""GPU: a captured call keeps the workspace its graph refers to when a later call or reservation needs a
larger one. Replayed after that, with other lengths, it matches the eager call bit for bit."""
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
from paged_decode_attention_kv_gb300 import workloads as wl
from test_gpu_decode import dev, dev_bits
from test_oracle_multi import Multi

pytestmark = pytest.mark.gpu


class Job:
    """A call without weights: one token (T = 0) or several, on the paged cache or the ring, with or
    without the rotary embedding."""

    def __init__(self, T, lens, seed, ring=0, rope=False):
        n = max(T, 1)
        m = Multi(seed, 64, 8, lens, [min(n, L) for L in lens], n)
        pick = (lambda x: x) if T else (lambda x: x[:, 0].contiguous())
        self.T, self.ring, self.scale = T, ring, m.c.scale
        self.q, self.kn, self.vn = (pick(dev_bits(x)) for x in (m.q, m.k_new, m.v_new))
        k, v = m.ring(ring) if ring else m.paged(1)[:2]
        self.k, self.v = dev_bits(k), dev_bits(v)
        self.bt = None if ring else dev(m.paged(1)[2])
        self.lens, self.n, self.sinks = dev(m.lens), dev(m.n), dev(m.sinks)
        self.rope = ()
        if rope:
            angle = torch.arange(max(lens) + 1, device="cuda")[:, None] / 100.0 ** (torch.arange(32, device="cuda") / 32)
            self.rope = (angle.cos().float().contiguous(), angle.sin().float().contiguous())
        self.out = torch.empty_like(self.q)

    def call(self, k, v, out):
        where, kw = () if self.ring else (self.bt,), {}
        name = "decode_attn_" + ("ring" if self.ring else "paged") + ("_multi" if self.T else "") + ("_rope" if self.rope else "")
        if self.T:
            kw["q_lens"] = self.n
        window = () if self.ring else (0,)
        getattr(da, name)(self.q, self.kn, self.vn, k, v, *where, self.lens, self.sinks, *self.rope, *window, self.scale, out, **kw)


@pytest.mark.parametrize("T,ring,rope,lens,later", [
    (0, 0, False, [300, 40, 90], [250, 37, 80]),
    (0, 128, False, [300, 40, 90], [250, 37, 80]),
    (0, 0, True, [300, 40, 90], [250, 37, 80]),
    (3, 0, False, [300, 40, 90], [250, 37, 80]),             # the decode kernel: partials and counters
    (5, 0, False, [6000, 40, 900], [5000, 37, 80]),          # 40 rows, split keys
    (5, 128, True, [300, 40, 90], [250, 37, 80]),            # the rotated rows
    (16, 0, False, [6000, 40, 900], [5000, 37, 80]),         # tcgen05, split keys, folded by a kernel of its own
    (5, 0, True, [6000, 40, 900], [5000, 37, 80])])
@pytest.mark.parametrize("grow", ["call", "weights", "reserve"])
def test_graph_outlives_its_workspace(T, ring, rope, lens, later, grow):
    job = Job(T, lens, 3000 + T, ring, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    da.decode_attn_stream_reserve(s)
    try:
        with torch.cuda.stream(s):
            job.call(job.k.clone(), job.v.clone(), torch.empty_like(job.out))
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                job.call(job.k, job.v, job.out)
            if grow == "reserve":
                da.decode_attn_stream_reserve(s, 1 << 26, 1 << 28)
            else:                                            # 64 tokens of 5 slots: many more row blocks and splits
                big = Job(64, [9000, 300, 7000, 64, 2000], 3100)
                if grow == "call":
                    big.call(big.k, big.v, big.out)
                else:
                    w = torch.zeros(big.k.shape[:3], device="cuda")
                    da.decode_attn_paged_multi_weights(big.q, big.kn, big.vn, big.k, big.v, w, big.bt, big.lens, None, 0, 0.125,
                                                       big.out, q_lens=big.n)
                da.decode_attn_stream_reserve(s, 1 << 26, 0)
            s.synchronize()
            junk = [torch.full((1 << 20,), 0x7fc00001, dtype=torch.int32, device="cuda") for _ in range(8)]
            job.lens.copy_(torch.tensor(later, dtype=torch.int32))
            k, v, out = job.k.clone(), job.v.clone(), torch.empty_like(job.out)
            for _ in range(2):                               # the second finds the counters as the first left them
                job.k.copy_(k)
                job.v.copy_(v)
                g.replay()
            job.call(k, v, out)
            s.synchronize()
        assert da.decode_attn_device_status(s) == 0
        assert torch.equal(job.out.view(torch.int16), out.view(torch.int16))
        for a, b in ((job.k, k), (job.v, v)):
            assert wl.bits(a).tobytes() == wl.bits(b).tobytes()
        del g, junk
    finally:
        da.decode_attn_stream_release(s)
