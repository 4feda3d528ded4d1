"""GPU parity of kv_evict / kv_evict_fp8 against the plain form: the kept cells, the new lengths,
and every byte of the caches and the weights (moved cells where they belong, all others as they
were), on weights with ties, zeros of both signs, infinities and NaN; and eviction together with
the calls that accumulate the weights and the attention that reads the smaller cache."""
import numpy as np
import pytest
import torch

import paged_decode_attention_kv_gb300 as da
import plain_weights as pw
from paged_decode_attention_kv_gb300 import workloads as wl
from test_gpu_decode import DEV, dev

pytestmark = pytest.mark.gpu


class Cache:
    """Random bytes behind a shuffled block table: bf16 pools or fp8 blocks, and weights."""

    def __init__(self, seed, Hkv, lens, fp8, width=None, kind="exp"):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        need = [-(-int(L) // 16) for L in lens]
        pages = sum(need) + 3
        perm = rng.permutation(pages).astype(np.int32)
        self.bt = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        self.fp8, self.Hkv = fp8, Hkv
        if fp8:
            self.kv = rng.integers(0, 256, (pages, Hkv, 2176), dtype=np.uint8)
        else:
            self.k = rng.integers(0, 65536, (pages, Hkv, 16, 64), dtype=np.uint16)
            self.v = rng.integers(0, 65536, (pages, Hkv, 16, 64), dtype=np.uint16)
        w = rng.exponential(size=(pages, Hkv, 16)) ** 3
        if kind == "ties":
            w = rng.integers(0, 4, w.shape)
        elif kind == "equal":
            w = np.full(w.shape, 0.25)
        elif kind == "zeros":
            w = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0)
        elif kind == "odd":
            w = rng.choice([0.0, -0.0, 1.0, 1.5, -2.0, 3.4e38, 1e-45, -1e-45, np.inf, -np.inf, np.nan, -np.nan], w.shape)
        self.w = w.astype(np.float32)

    def call(self, keep, first, last, max_seq_len=None, stream=None):
        B = len(self.lens)
        new_lens = torch.full((B,), -7, dtype=torch.int32, device=DEV)
        kept = torch.full((B, self.Hkv, keep), -7, dtype=torch.int32, device=DEV)
        w = dev(self.w)
        args = (w, dev(self.bt), dev(self.lens), new_lens, kept, first, last)
        if self.fp8:
            kv = dev(self.kv)
            da.kv_evict_fp8(kv, *args, max_seq_len=max_seq_len, stream=stream)
            pools = (kv.cpu().numpy(),)
        else:
            k, v = wl.from_bits(self.k, DEV), wl.from_bits(self.v, DEV)
            da.kv_evict(k, v, *args, max_seq_len=max_seq_len, stream=stream)
            pools = (wl.bits(k), wl.bits(v))
        return pools, w.cpu().numpy(), new_lens.cpu().numpy(), kept.cpu().numpy()

    def moved(self, kept, lens=None):
        lens = self.lens if lens is None else lens
        w = pw.move(self.w, self.bt, lens, kept)
        if not self.fp8:
            return (pw.move(self.k, self.bt, lens, kept), pw.move(self.v, self.bt, lens, kept)), w
        n, H = self.kv.shape[0], self.Hkv
        out = self.kv.copy()
        out[..., :1024] = pw.move(self.kv[..., :1024].reshape(n, H, 16, 64), self.bt, lens, kept).reshape(n, H, 1024)
        vt = self.kv[..., 1024:2048].reshape(n, H, 64, 16).transpose(0, 1, 3, 2)
        out[..., 1024:2048] = pw.move(vt, self.bt, lens, kept).transpose(0, 1, 3, 2).reshape(n, H, 1024)
        for o in (2048, 2112):
            out[..., o:o + 64] = pw.move(self.kv[..., o:o + 64].reshape(n, H, 16, 4), self.bt, lens, kept).reshape(n, H, 64)
        return (out,), w


def check(c, keep, first, last, status=0, **kw):
    pools, w, new_lens, kept = c.call(keep, first, last, **kw)
    assert da.decode_attn_device_status() == status
    want_kept, want_lens = pw.evict_maps(c.w, c.bt, c.lens, keep, first, last)
    np.testing.assert_array_equal(new_lens, want_lens)
    np.testing.assert_array_equal(kept, want_kept)
    want_pools, want_w = c.moved(want_kept)
    for a, b in zip(pools, want_pools):
        np.testing.assert_array_equal(a, b)
    np.testing.assert_array_equal(w.view(np.uint32), want_w.view(np.uint32))


LENS = [0, 1, 15, 16, 17, 33, 100, 257, 1000, 63, 64, 65]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (16, 4, 4), (17, 0, 16), (63, 1, 0), (64, 4, 33),
                                             (64, 32, 32), (99, 0, 0), (500, 4, 250), (1000, 4, 8), (2000, 0, 0)])
def test_every_byte(fp8, keep, first, last):
    """Budgets from one cell to more than any sequence has, first and last cells from none to all of
    it (nothing left to choose), tails that overlap the place they move to."""
    check(Cache(keep + first, 3, LENS, fp8), keep, first, last)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["ties", "equal", "zeros", "odd"])
def test_ties_zeros_infinities_and_nan(fp8, kind):
    c = Cache(40, 2, [500, 77, 300, 64], fp8, kind=kind)
    check(c, 60, 2, 5)
    check(c, 200, 0, 0)
    check(c, 299, 7, 101)


@pytest.mark.parametrize("L,keep,last", [(4160, 4096, 256), (4097, 4096, 4096), (4097, 4096, 0), (9000, 100, 7), (30000, 8192, 512),
                                         (30000, 29999, 20000), (20001, 20000, 9)])
@pytest.mark.parametrize("B,Hkv", [(1, 1), (1, 8), (3, 2)])
def test_long_sequences_over_clusters(L, keep, last, B, Hkv):
    c = Cache(L + keep + B, Hkv, [L - 3 * i for i in range(B)], False)
    check(c, keep, min(4, keep - last), last)


def test_fp8_long():
    check(Cache(77, 2, [9001, 4100], True), 4096, 4, 700)


def test_keys_beyond_shared_memory():
    """A sequence longer than the shared memory of a cluster: the weights are read again each round."""
    c = Cache(5, 1, [420001], False, kind="ties")
    check(c, 5000, 4, 100)


def test_batch_of_many_slots():
    rng = np.random.default_rng(6)
    lens = [0 if rng.random() < 0.2 else int(rng.integers(1, 900)) for _ in range(300)]
    check(Cache(6, 4, lens, False), 128, 4, 32)
    check(Cache(7, 1, [int(x) for x in rng.integers(1, 60, 1024)], False), 20, 1, 5)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_lengths(fp8):
    """Cells of a page outside the pool rank lowest; where they are kept all the same, the moves into
    and out of them are skipped. A bad length is an inactive slot."""
    c = Cache(8, 2, [200, 300, 90], fp8)
    c.bt[0, 3], c.bt[1, 17], c.bt[1, 18] = -1, c.w.shape[0], 2 ** 31 - 1
    check(c, 100, 4, 20, status=da.DA_STATUS_BAD_PAGE)
    check(c, 199, 4, 20, status=da.DA_STATUS_BAD_PAGE)
    c = Cache(9, 2, [200, 300, 90], fp8)
    true_lens = c.lens
    c.lens = np.asarray([-5, 300, 305], np.int32)
    pools, w, new_lens, kept = c.call(100, 4, 20)
    assert da.decode_attn_device_status() == da.DA_STATUS_BAD_SEQ_LEN
    assert new_lens.tolist() == [0, 100, 0] and np.all(kept[[0, 2]] == -1)
    c.lens = np.asarray([0, 300, 0], np.int32)
    want, _ = pw.evict_maps(c.w, c.bt, c.lens, 100, 4, 20)
    np.testing.assert_array_equal(kept, want)
    for a, b in zip(pools, c.moved(want)[0]):
        np.testing.assert_array_equal(a, b)
    c.lens = np.asarray([200, 300, 90], np.int32)
    pools, w, new_lens, kept = c.call(100, 4, 20, max_seq_len=250)   # one length beyond the bound
    assert da.decode_attn_device_status() == da.DA_STATUS_BAD_SEQ_LEN
    assert new_lens.tolist() == [100, 0, 90]


def test_refusals():
    c = Cache(10, 2, [200, 90], False)
    k, v, w, bt, sl = wl.from_bits(c.k, DEV), wl.from_bits(c.v, DEV), dev(c.w), dev(c.bt), dev(c.lens)
    nl, kept = torch.zeros_like(sl), torch.zeros((2, 2, 50), dtype=torch.int32, device=DEV)
    for name, args in (("kept", (k, v, w, bt, sl, nl, kept[:, :, ::2])), ("kept", (k, v, w, bt, sl, nl, kept[:1])),
                       ("new_lens", (k, v, w, bt, sl, nl.long(), kept)), ("weights", (k, v, w.half(), bt, sl, nl, kept)),
                       ("v_cache", (k, v[:3], w, bt, sl, nl, kept))):
        with pytest.raises(ValueError, match=name):
            da.kv_evict(*args)
    for args, kw in (((sl, kept), dict()), ((nl, kept), dict(keep_first=-1)), ((nl, kept), dict(keep_first=30, keep_last=21)),
                     ((nl, kept[:, :, :0].contiguous()), dict())):
        with pytest.raises(da.DecodeAttnError) as e:
            da.kv_evict(k, v, w, bt, sl, *args, **kw)
        assert e.value.code == -1
    assert torch.equal(k.view(torch.int16), wl.from_bits(c.k, DEV).view(torch.int16))


def test_graph_replay_and_repeated_calls():
    """A captured eviction replayed with other lengths and weights; repeated calls are identical."""
    c = Cache(11, 4, [700, 200, 90, 1500], False, width=120)
    k, v, w, bt, sl = wl.from_bits(c.k, DEV), wl.from_bits(c.v, DEV), dev(c.w), dev(c.bt), dev(c.lens)
    nl, kept = torch.zeros_like(sl), torch.zeros((4, 4, 150), dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    da.decode_attn_weights_reserve(da.kv_evict_workspace_bytes(4, 4, 150))
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            da.kv_evict(k, v, w, bt, sl, nl, kept, 4, 30)
    s.synchronize()
    for lens in ([700, 200, 90, 1500], [151, 150, 90, 1000]):
        c.lens = np.asarray(lens, np.int32)
        for t, a in ((k, c.k), (v, c.v)):
            t.copy_(wl.from_bits(a, DEV))
        w.copy_(dev(c.w))
        sl.copy_(dev(c.lens))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want, want_lens = pw.evict_maps(c.w, c.bt, c.lens, 150, 4, 30)
        np.testing.assert_array_equal(kept.cpu().numpy(), want)
        np.testing.assert_array_equal(nl.cpu().numpy(), want_lens)
        (wk, wv), ww = c.moved(want)
        np.testing.assert_array_equal(wl.bits(k), wk)
        np.testing.assert_array_equal(wl.bits(v), wv)
        np.testing.assert_array_equal(w.cpu().numpy().view(np.uint32), ww.view(np.uint32))
        c.w = np.random.default_rng(12).random(c.w.shape).astype(np.float32)


@pytest.mark.parametrize("level", [0, 1, 2])
def test_the_next_call_reads_the_new_lengths(level):
    """An eviction and an attention call on its new_lens right behind it, at every early-input level
    (the early levels read the lengths before they wait for the kernel before): the same output
    as with a wait between the two, every time. The lengths start as ones, so that a stale
    read shows."""
    c = Cache(13, 2, [700, 300, 1500, 64], False, width=120)
    w0, bt, sl = dev(c.w), dev(c.bt), dev(c.lens)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    pages = c.k.shape[0]
    k0, v0 = (torch.randn((pages, 2, 16, 64), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((4, 16, 64), generator=gen, device=DEV).to(torch.bfloat16)
    kept = torch.zeros((4, 2, 150), dtype=torch.int32, device=DEV)

    def run(wait):
        k, v, w = k0.clone(), v0.clone(), w0.clone()
        nl, out = torch.ones_like(sl), torch.empty_like(q)
        torch.cuda.synchronize()
        da.kv_evict(k, v, w, bt, sl, nl, kept, 4, 30)
        if wait:
            torch.cuda.synchronize()
        da.decode_attn_paged(q, None, None, k, v, bt, nl, None, 0, 0.125, out)
        torch.cuda.synchronize()
        return out

    prev = da.decode_attn_set_early_inputs(level)
    try:
        want = run(True)
        for _ in range(10):
            assert torch.equal(run(False).view(torch.int16), want.view(torch.int16))
    finally:
        da.decode_attn_set_early_inputs(prev)
    assert da.decode_attn_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_decode_under_a_budget(fp8):
    """The calls as an engine uses them: a prompt with weights (bf16), decode steps that append and
    accumulate, an eviction every few steps, the next steps on the smaller cache. A float64 model
    follows the tokens each KV head holds; the output of every step within the attention
    tolerance, and the kept cells equal wherever the model's weights are not within rounding of
    each other (their margin is checked, not assumed)."""
    gen = wl.cpu_generator(99)
    B, Hq, Hkv, D, keep, first, last = 3, 16, 2, 64, 96, 4, 24
    G, pages = Hq // Hkv, 64
    prompt = [150, 40, 97]
    bt = np.arange(B * 20, dtype=np.int32).reshape(B, 20)
    w = torch.zeros((pages, Hkv, 16), dtype=torch.float32, device=DEV)
    btd, lens = dev(bt), torch.zeros(B, dtype=torch.int32, device=DEV)
    T = max(prompt)
    keys = [[[] for _ in range(Hkv)] for _ in range(B)]      # the model: (k, v, weight) of each cell
    if fp8:
        kv = torch.zeros((pages, Hkv, 2176), dtype=torch.uint8, device=DEV)
    else:
        kc, vc = (torch.zeros((pages, Hkv, 16, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def stored(x):
        """A row as the cache holds it, in 64 bits."""
        if not fp8:
            return x.double().numpy()
        top = x.float().abs().amax(-1, keepdim=True)
        sc = torch.where(top > 0, top * torch.tensor(np.float32(1) / np.float32(448)), torch.ones_like(top))
        return ((x.float() / sc).to(torch.float8_e4m3fn).double() * sc.double()).numpy()

    def attend(b, q, n):
        """Model step of one sequence: q [n, Hq, D]; its last n cells are the new tokens."""
        out = np.zeros((n, Hq, D))
        for g in range(Hkv):
            cells = keys[b][g]
            L = len(cells)
            K, V = np.stack([c[0] for c in cells])[:, None], np.stack([c[1] for c in cells])[:, None]
            o, mass, _ = pw.step(q[:, g * G:(g + 1) * G], K, V, L, n, None, 0, 0.125)
            out[:, g * G:(g + 1) * G] = o
            for j in range(L):
                cells[j][2] = mass[j, 0] if j >= L - n else cells[j][2] + mass[j, 0]
        return out

    def agree(got, want):
        assert np.all(np.abs(got - want) <= 4e-3 + 1e-2 * np.abs(want))

    def append(b, kn, vn):
        for g in range(Hkv):
            keys[b][g].append([stored(kn[g]), stored(vn[g]), 0.0])

    if not fp8:
        q, kn, vn = (wl.randn_bf16((B, T, h, D), gen) for h in (Hq, Hkv, Hkv))
        for b in range(B):
            for t in range(prompt[b]):
                append(b, kn[b, t], vn[b, t])
        lens.copy_(torch.tensor(prompt, dtype=torch.int32))
        out = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=DEV)
        da.decode_attn_paged_multi_weights(dev(q), dev(kn), dev(vn), kc, vc, w, btd, lens, None, 0, 0.125, out, q_lens=lens)
        for b in range(B):
            agree(out[b, :prompt[b]].double().cpu().numpy(), attend(b, q[b, :prompt[b]].double().numpy(), prompt[b]))
    evictions = 0
    for step in range(140 if fp8 else 60):
        q, kn, vn = (wl.randn_bf16((B, h, D), gen) for h in (Hq, Hkv, Hkv))
        lens += 1
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=DEV)
        if fp8:
            da.decode_attn_paged_fp8_weights(dev(q), dev(kn), dev(vn), kv, w, btd, lens, None, 0, 0.125, out)
        else:
            da.decode_attn_paged_weights(dev(q), dev(kn), dev(vn), kc, vc, w, btd, lens, None, 0, 0.125, out)
        for b in range(B):
            append(b, kn[b], vn[b])
            agree(out[b].double().cpu().numpy(), attend(b, q[b][None].double().numpy(), 1)[0])
        if step % 16 == 15:
            new_lens, kept = torch.empty_like(lens), torch.empty((B, Hkv, keep), dtype=torch.int32, device=DEV)
            if fp8:
                da.kv_evict_fp8(kv, w, btd, lens, new_lens, kept, first, last)
            else:
                da.kv_evict(kc, vc, w, btd, lens, new_lens, kept, first, last)
            got = kept.cpu().numpy()
            for b in range(B):
                for g in range(Hkv):
                    cells = keys[b][g]
                    L = len(cells)
                    if L <= keep:
                        assert got[b, g].tolist() == list(range(L)) + [-1] * (keep - L)
                        continue
                    evictions += 1
                    wt = np.array([c[2] for c in cells])
                    mid = np.sort(wt[first:L - last])[::-1]
                    n = keep - first - last
                    if n < len(mid):  # the model's choice is clear of the rounding of both sides
                        assert mid[n - 1] - mid[n] > 1e-4 * mid[n]
                    want = pw.kept_cells(wt, L, keep, first, last)
                    assert got[b, g].tolist() == want.tolist()
                    keys[b][g] = [cells[i] for i in want]
            lens = new_lens
            assert lens.tolist() == [len(keys[b][0]) for b in range(B)]
    torch.cuda.synchronize()
    assert da.decode_attn_device_status() == 0
    assert evictions >= 8
