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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("level", [0, 1, 2])
def test_graphs_that_share_the_workspaces(fp8, level):
    """A step with weights, a chunk with weights (bf16), an eviction by clusters and a step on the evicted
    cache, a graph each, captured on one stream and so on the same workspaces: replayed in turn, twice,
    they leave what the eager calls leave, bit for bit."""
    gen = wl.cpu_generator(5000 + level)
    B, Hq, Hkv, T, keep, pages = 2, 64, 8, 12, 500, 1300
    lens = torch.tensor([9000, 8500], dtype=torch.int32)
    table = torch.randperm(pages, generator=gen)[:2 * 600].to(torch.int32).view(2, 600)
    bt, l1, l2 = dev(table), dev(lens), dev(lens + T)
    q, kn, vn = (dev(wl.randn_bf16((B, h, 64), gen)) for h in (Hq, Hkv, Hkv))
    qt, knt, vnt = (dev(wl.randn_bf16((B, T, h, 64), gen)) for h in (Hq, Hkv, Hkv))
    if fp8:
        kv = torch.randint(0, 256, (pages, Hkv, 2176), generator=gen, dtype=torch.uint8)
        kv[..., :2048][(kv[..., :2048] & 127) == 127] = 0
        kv[..., 2048:] = torch.full((pages, Hkv, 32), 0.005).view(torch.uint8)
        first = [dev(kv)]
    else:
        first = [dev(wl.randn_bf16((pages, Hkv, 16, 64), gen)) for _ in range(2)]
    first.append(torch.rand((pages, Hkv, 16), device="cuda"))

    def state():
        return [x.clone() for x in first] + [torch.zeros_like(l1), torch.zeros((B, Hkv, keep), dtype=torch.int32, device="cuda"),
                                             torch.zeros_like(q), torch.zeros_like(qt), torch.zeros_like(q)]

    def calls(s):
        *pools, w, nl, kept, o1, ot, o2 = s
        f = "_fp8" if fp8 else ""
        yield lambda: getattr(da, f"decode_attn_paged{f}_weights")(q, kn, vn, *pools, w, bt, l1, None, 0, 0.125, o1)
        if not fp8:
            yield lambda: da.decode_attn_paged_multi_weights(qt, knt, vnt, *pools, w, bt, l2, None, 0, 0.125, ot)
        yield lambda: getattr(da, "kv_evict" + f)(*pools, w, bt, l1 if fp8 else l2, nl, kept, 4, 64)
        yield lambda: getattr(da, "decode_attn_paged" + f)(q, None, None, *pools, bt, nl, None, 0, 0.125, o2)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    da.decode_attn_stream_reserve(s)
    prev = da.decode_attn_set_early_inputs(level)
    try:
        with torch.cuda.stream(s):
            eager, replayed, graphs = state(), state(), []
            for _ in range(2):
                for f in calls(eager):
                    f()
            s.synchronize()
            for f in calls(replayed):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    f()
                graphs.append(g)
            for _ in range(2):
                for g in graphs:
                    g.replay()
            s.synchronize()
        assert da.decode_attn_device_status(s) == 0
        for i, (a, b) in enumerate(zip(eager, replayed)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
        assert replayed[-5].tolist() == [keep, keep]
        del graphs
    finally:
        da.decode_attn_set_early_inputs(prev)
        da.decode_attn_stream_release(s)
