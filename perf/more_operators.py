"""A step of new tokens over the fp8 cache, from the projection's output to the attention, as measured cases.

  rotate  queries and keys of packed projection rows: the RMS norm of each head (with weights, or none) and the rotary
          rotation at given positions of one or several axes (time, height, width); the value rows are copied
  store   the new tokens of every sequence quantised into fp8 blocks (paged, or a ring), and positions from `start` on
          read back as bf16
  attend  several new tokens per sequence: quantised into their pages, then causal attention of their query rows over
          the fp8 pages

Layouts are the framework's: fp8 blocks [pages, Hkv, 2176] (16 tokens: K codes [16][64], V codes [64][16], K scales, V
scales), block tables [B, max pages], lengths counted after the append (0 = inactive slot). A row's scale is its largest
magnitude / 448, a 32-bit division (1 for a row of zeros), and a code the e4m3 value nearest to x / scale.
"""
import math
import random

import torch

own = False

PAGE, D, HALF = 16, 64, 32
SCALE = 0.125
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's decode step, latency counts: per-head norms and the rotation
        dict(name="rotate_b1", op="rotate", tokens=1, hq=64, hkv=8, norm=True, axes=1, order="blocks", span=131072),
        # the batch-64 decode step
        dict(name="rotate_b64", op="rotate", tokens=64, hq=64, hkv=8, norm=True, axes=1, order="blocks", span=8192),
        # prompts of 8191 tokens of text, images and video: three axes
        dict(name="rotate_axes", op="rotate", tokens=8191, hq=64, hkv=8, norm=True, axes=3, order="blocks", span=8192),
        # the batch-64 decode step's tokens written, and what was written read back
        dict(name="store_b64", op="store", batch=64, hkv=8, lens="uniform", lo=1024, hi=8192, inactive=0, tokens=1, counts="full", ring=0, back="new"),
        # whole prompts of several users written and read back
        dict(name="store_prompts", op="store", batch=16, hkv=8, lens="uniform", lo=1201, hi=4096, inactive=0, tokens=4096, counts="whole", ring=0, back="all"),
        # a long cached prefix handed to code that wants bf16, behind an append of one chunk
        dict(name="store_long1", op="store", batch=1, hkv=8, lens="fixed", lo=131072, hi=131072, inactive=0, tokens=512, counts="full", ring=0, back="all"),
        # draft verification: up to four new tokens per sequence
        dict(name="attend_verify", op="attend", batch=32, hq=64, hkv=8, lens="uniform", lo=1024, hi=8192, inactive=0, window=0, sinks=True, tokens=4, counts="ragged"),
        # draft verification behind one very long history
        dict(name="attend_long1", op="attend", batch=1, hq=64, hkv=8, lens="fixed", lo=131072, hi=131072, inactive=0, window=0, sinks=True, tokens=4, counts="full"),
        # long drafts (or short chunks) of the batch-64 step
        dict(name="attend_b64", op="attend", batch=64, hq=64, hkv=8, lens="uniform", lo=1024, hi=8192, inactive=0, window=0, sinks=True, tokens=16, counts="full"),
        # a chunk of a prompt behind its history
        dict(name="attend_chunk", op="attend", batch=1, hq=64, hkv=8, lens="fixed", lo=8192, hi=8192, inactive=0, window=0, sinks=True, tokens=512, counts="full"),
        # whole prompts of several users, of different lengths
        dict(name="attend_fresh", op="attend", batch=4, hq=64, hkv=8, lens="uniform", lo=1201, hi=2048, inactive=0, window=0, sinks=True, tokens=2048, counts="whole"),
        # serving slots of very different lengths, some inactive, four query heads per KV head, a window that starts inside a page
        dict(name="attend_slots", op="attend", batch=48, hq=32, hkv=8, lens="lognormal", lo=9, hi=16384, inactive=12, window=4001, sinks=False, tokens=9, counts="ragged"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "store", "attend", "attend"])
    g = rng.choice([1, 2, 4, 8, 8, 16])
    hkv = rng.choice([1, 2, 4, 8, 8, 12])
    if op == "rotate":
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, tokens=_log_int(rng, 1, max(1, 2 ** 19 // ((g + 2) * hkv))), hq=g * hkv, hkv=hkv, norm=rng.random() < 0.7, axes=axes,
                    order=rng.choice(["blocks", "turns"]) if axes > 1 else "blocks", span=_log_int(rng, 64, 131072))
    if op == "store":
        t = _log_int(rng, 1, 4096)
        hi = _log_int(rng, t, 65536)
        b = max(1, min(_log_int(rng, 1, 128), 2 ** 19 // (hkv * hi), 2 ** 18 // hi))
        ring = rng.choice([0, 0, 16 * _log_int(rng, 1, 256)])
        return dict(op=op, batch=b, hkv=hkv, lens=rng.choice(["fixed", "uniform", "lognormal"]), lo=max(1, hi // 7), hi=hi, inactive=rng.choice([0, 0, b // 4]),
                    tokens=t, counts=rng.choice(["full", "ragged"]), ring=ring, back=rng.choice(["new", "all"]))
    t = _log_int(rng, 1, 1024)
    pairs = 2 ** 27 // max(64, g * hkv)  # (new token, position) pairs over the batch at most
    hi = max(t + 1, _log_int(rng, 64, max(128, min(65536, pairs // t))))
    b = max(1, min(_log_int(rng, 1, 64), pairs // (t * hi), 2 ** 18 // hi))
    return dict(op=op, batch=b, hq=g * hkv, hkv=hkv, lens=rng.choice(["fixed", "uniform", "lognormal"]), lo=max(1, hi // 5), hi=hi, inactive=rng.choice([0, 0, b // 4]),
                window=rng.choice([0, 0, _log_int(rng, 1, hi)]), sinks=rng.random() < 0.7, tokens=t, counts=rng.choice(["full", "ragged"]))


def _lens(c):
    """The lengths of a case: the same for every seed, so that its work is too."""
    rng = random.Random("%d %d %d %s" % (c["batch"], c["lo"], c["hi"], c["lens"]))
    n = c["batch"]
    if c["lens"] == "fixed":
        lens = [c["hi"]] * n
    elif c["lens"] == "uniform":
        lens = [rng.randint(c["lo"], c["hi"]) for _ in range(n)]
    else:  # lognormal, its median an eighth of the longest
        lens = [min(c["hi"], max(c["lo"], 1, math.ceil(c["hi"] / 8 * math.exp(rng.gauss(0, 1))))) for _ in range(n)]
    for i in rng.sample(range(n), c["inactive"]):
        lens[i] = 0
    return lens


def _counts(c, lens):
    """New tokens per sequence."""
    rng = random.Random("%d %s" % (c["tokens"], c["counts"]))
    return [min(L, rng.randint(1, c["tokens"]) if c["counts"] == "ragged" else c["tokens"]) for L in lens]


def _sections(c):
    """Pairs per axis, and the axis of each of the 32 pairs: in blocks, or the axes taking turns."""
    sections = {1: (32,), 2: (12, 20), 3: (8, 12, 12)}[c["axes"]]
    if c["order"] == "blocks":
        return sections, [a for a, n in enumerate(sections) for _ in range(n)]
    left, axis, a = list(sections), [], 0
    while len(axis) < HALF:
        if left[a]:
            left[a] -= 1
            axis.append(a)
        a = (a + 1) % len(sections)
    return sections, axis


def _back(c, lens, counts):
    """The first position read back of every sequence, and the most positions of one."""
    starts = []
    for L, n in zip(lens, counts):
        s = L - n if c["back"] == "new" else 0
        starts.append(max(s, L - c["ring"]) if c["ring"] else s)
    return starts, max(1, max(L - s for L, s in zip(lens, starts)))


# ---------------------------------------------------------------- inputs
class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=torch.float32)

    def ints(self, hi, *shape):
        return torch.randint(0, hi, shape, generator=self.g, device="cuda", dtype=torch.int32)

    def blocks(self, *lead):
        """fp8 blocks: finite e4m3 codes of both signs, and scales of rows whose largest value is 2 to 3."""
        codes = torch.randint(0, 256, lead + (2 * PAGE * D,), generator=self.g, device="cuda", dtype=torch.uint8)
        codes = torch.where((codes & 127) == 127, codes - 1, codes)
        scales = (2 + self.uniform(*lead, 2 * PAGE)) / 448
        return torch.cat([codes, scales.view(torch.uint8)], -1).contiguous()


def _positions(r, c):
    """[axes, N]: running positions of the tokens, and (several axes) frames, rows and columns of a picture within them."""
    n, span = c["tokens"], c["span"]
    at = torch.arange(n, device="cuda", dtype=torch.int32)
    first = int(r.ints(span, 1).item())
    rows = [(first + at) % span]
    for a in range(1, c["axes"]):
        rows.append((first + at // (1, 32, 1)[a] % 32) % span)
    return torch.stack(rows).contiguous()


def prepare(case, seed):
    c, r = case, _Draw(seed)
    if c["op"] == "rotate":
        n, heads = c["tokens"], c["hq"] + 2 * c["hkv"]
        qkv = r.normal(n, heads, D)
        angle = torch.arange(c["span"], device="cuda", dtype=torch.float64)[:, None] * 150000.0 ** (-torch.arange(HALF, device="cuda", dtype=torch.float64) / HALF)
        s = dict(case=c, q=qkv[:, : c["hq"]], k=qkv[:, c["hq"] : c["hq"] + c["hkv"]], v=qkv[:, c["hq"] + c["hkv"] :], positions=_positions(r, c),
                 rope_cos=angle.cos().float().contiguous(), rope_sin=angle.sin().float().contiguous())
        s["q_weight"], s["k_weight"] = (0.5 + r.uniform(D), 0.5 + r.uniform(D)) if c["norm"] else (None, None)
        for x in "qkv":
            s[x + "_out"] = torch.empty(s[x].shape, dtype=torch.bfloat16, device="cuda")
        return s
    lens = _lens(c)
    counts = _counts(c, lens)
    B, hkv = c["batch"], c["hkv"]
    s = dict(case=c, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q_lens=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    if c.get("ring"):
        s["kv_cache"], s["block_table"] = r.blocks(B, hkv, c["ring"] // PAGE), None
    else:
        need = [-(-L // PAGE) for L in lens]
        pages, cols = max(1, sum(need) + sum(need) // 10), max(1, max(need))
        perm = torch.randperm(pages, generator=r.g, device="cuda").to(torch.int32)
        n, at = torch.tensor(need, device="cuda"), torch.arange(cols, device="cuda")[None, :]
        s["block_table"] = torch.where(at < n[:, None], perm[((n.cumsum(0) - n)[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
        s["kv_cache"] = r.blocks(pages, hkv)
    s["k_new"], s["v_new"] = r.normal(B, c["tokens"], hkv, D), r.normal(B, c["tokens"], hkv, D)
    if c["op"] == "attend":
        s["q"] = r.normal(B, c["tokens"], c["hq"], D)
        s["sinks"] = r.normal(c["hq"]).float() if c["sinks"] else None
        s["out"] = torch.empty_like(s["q"])
    else:
        starts, rows = _back(c, lens, counts)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["k_out"], s["v_out"] = (torch.zeros((B, rows, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return s


# ---------------------------------------------------------------- the plain forms
def _plain_rotate(s):
    axis = torch.tensor(_sections(s["case"])[1], device="cuda")
    pos = s["positions"].long()[axis].T                                    # [N, 32] each pair's position
    pair = torch.arange(HALF, device="cuda")
    c, sn = s["rope_cos"][pos, pair][:, None], s["rope_sin"][pos, pair][:, None]
    for x in "qk":
        y = s[x].float()
        if s[x + "_weight"] is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s[x + "_weight"]
        a, b = y[..., :HALF], y[..., HALF:]
        s[x + "_out"].copy_(torch.cat([a * c - b * sn, b * c + a * sn], -1))
    s["v_out"].copy_(s["v"])


def _quantise(x):
    """e4m3 codes (as bytes) and the scale of each row."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / torch.full_like(top, 448), torch.ones_like(top))
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale[..., 0]


def _new(s):
    """Sequence, index and position of every new token that is stored (a ring keeps the last ones)."""
    c, n, L = s["case"], s["q_lens"].long(), s["seq_lens"].long()
    t = torch.arange(c["tokens"], device="cuda")
    keep = t[None, :] < n[:, None]
    pos = (L - n)[:, None] + t
    if c.get("ring"):
        keep = keep & (pos >= (L - c["ring"])[:, None])
    b, t = keep.nonzero(as_tuple=True)
    return b, t, pos[b, t]


def _block(s, b, pos):
    """Index of the block of position pos[N] of sequence b[N] among blocks of Hkv heads, and the stride of a head."""
    c = s["case"]
    if c.get("ring"):
        per = c["ring"] // PAGE
        return b * c["hkv"] * per + pos % c["ring"] // PAGE, per
    return s["block_table"].long()[b, pos // PAGE] * c["hkv"], 1


def _store(s):
    b, t, pos = _new(s)
    (kc, ks), (vc, vs) = _quantise(s["k_new"][b, t]), _quantise(s["v_new"][b, t])
    first, step = _block(s, b, pos)
    h, d = torch.arange(s["case"]["hkv"], device="cuda"), torch.arange(D, device="cuda")
    kv = s["kv_cache"].view(-1, s["kv_cache"].shape[-1])
    blk = first[:, None] + h * step                                        # [N, Hkv]
    sl = (pos % PAGE)[:, None]
    kv[blk[..., None], sl[..., None] * D + d] = kc
    kv[blk[..., None], PAGE * D + d * PAGE + sl[..., None]] = vc
    scales = kv.view(torch.float32)[:, 2 * PAGE * D // 4 :]
    scales[blk, sl] = ks
    scales[blk, PAGE + sl] = vs


def _split(kv):
    """Views of fp8 blocks: K codes [.., 16, 64], V codes [.., 64, 16], K scales, V scales [.., 16]."""
    n = PAGE * D
    codes = kv[..., : 2 * n].view(torch.float8_e4m3fn)
    scales = kv[..., 2 * n :].view(torch.float32)
    return codes[..., :n].unflatten(-1, (PAGE, D)), codes[..., n:].unflatten(-1, (D, PAGE)), scales[..., :PAGE], scales[..., PAGE:]


def _plain_read(s):
    at = s["starts"].long()[:, None] + torch.arange(s["k_out"].shape[1], device="cuda")
    b, i = (at < s["seq_lens"].long()[:, None]).nonzero(as_tuple=True)
    pos = at[b, i]
    first, step = _block(s, b, pos)
    h, d = torch.arange(s["case"]["hkv"], device="cuda"), torch.arange(D, device="cuda")
    kv = s["kv_cache"].view(-1, s["kv_cache"].shape[-1])
    blk = first[:, None] + h * step                                        # [N, Hkv]
    sl = (pos % PAGE)[:, None]
    scales = kv.view(torch.float32)[:, 2 * PAGE * D // 4 :]
    k = kv[blk[..., None], sl[..., None] * D + d].view(torch.float8_e4m3fn).float() * scales[blk, sl][..., None]
    v = kv[blk[..., None], PAGE * D + d * PAGE + sl[..., None]].view(torch.float8_e4m3fn).float() * scales[blk, PAGE + sl][..., None]
    s["k_out"][b, i], s["v_out"][b, i] = k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_attend(s):
    c, bt = s["case"], s["block_table"]
    _store(s)  # the new tokens first: every key is then read from the cache
    x = s["kv_cache"][bt.clamp(min=0).long()]
    k, v, ks, vs = _split(x)
    k = (k.float() * ks[..., None]).transpose(1, 2).flatten(2, 3)          # [B, Hkv, cells, D]
    v = (v.float().transpose(-1, -2) * vs[..., None]).transpose(1, 2).flatten(2, 3)
    T = c["tokens"]
    q = s["q"].view(c["batch"], T, c["hkv"], -1, D)
    B, _, H, G, _ = q.shape
    L, n = s["seq_lens"].long(), s["q_lens"].long()
    t, j = torch.arange(T, device="cuda"), torch.arange(bt.shape[1] * PAGE, device="cuda")
    p = ((L - n)[:, None] + t)[:, :, None]                                 # [B, T, 1] each query's position
    see = (j <= p) & (t[None, :, None] < n[:, None, None])
    if c["window"]:
        see = see & (j > p - c["window"])
    x = torch.matmul(q.float().permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D), k.transpose(2, 3)).mul_(SCALE)
    x = x.view(B, H, T, G, -1).masked_fill_(~see[:, None, :, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, H, 1, G, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    den = x.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        den = den + torch.exp(sink - top)
    x = x.div_(torch.where(den > 0, den, torch.ones_like(den)))
    v = torch.where((j < L[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(x.view(B, H, T * G, -1), v).view(B, H, T, G, D).permute(0, 2, 1, 3, 4)
    real = (t < n[:, None])[:, :, None, None]
    s["out"].copy_(torch.where(real, o.reshape(s["out"].shape), torch.zeros((), device="cuda")))


def _cache(s):
    n = 2 * PAGE * D
    return dict(codes=s["kv_cache"][..., :n].view(torch.float8_e4m3fn), scales=s["kv_cache"][..., n:].view(torch.float32))


def run(state):
    s, c = state, state["case"]
    if own:
        import paged_decode_attention_kv_gb300 as da
    if c["op"] == "rotate":
        if own:
            da.qk_norm_rope(s["q"], s["k"], s["positions"], s["rope_cos"], s["rope_sin"], s["q_out"], s["k_out"], q_weight=s["q_weight"],
                            k_weight=s["k_weight"], eps=EPS, sections=_sections(c)[0], interleaved=c["order"] == "turns", v=s["v"], v_out=s["v_out"])
        else:
            _plain_rotate(s)
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    if c["op"] == "store":
        if own:
            da.kv_append_fp8(s["k_new"], s["v_new"], s["kv_cache"], s["seq_lens"], s["block_table"], q_lens=s["q_lens"])
            da.kv_read_fp8(s["kv_cache"], s["seq_lens"], s["k_out"], s["v_out"], s["block_table"], starts=s["starts"])
        else:
            _store(s)
            _plain_read(s)
        return dict(_cache(s), k=s["k_out"], v=s["v_out"])
    if own:
        da.decode_attn_paged_fp8_multi(s["q"], s["k_new"], s["v_new"], s["kv_cache"], s["block_table"], s["seq_lens"], s["sinks"], c["window"], SCALE,
                                       s["out"], q_lens=s["q_lens"])
    else:
        _plain_attend(s)
    return dict(_cache(s), out=s["out"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rotate":
        n, rows = c["tokens"], c["hq"] + 2 * c["hkv"]
        tables = 8 * HALF * min(n, c["span"])
        return dict(bytes=n * rows * 4 * D + 4 * n * c["axes"] + tables, flops=n * (c["hq"] + c["hkv"]) * D * (7 if c["norm"] else 3))
    lens = _lens(c)
    counts = _counts(c, lens)
    hkv, token = c["hkv"], 2 * D + 8  # bytes of K and V of one token and KV head
    if c["op"] == "store":
        starts, _ = _back(c, lens, counts)
        new = sum(min(n, c["ring"] or n) for n in counts)
        fresh = sum(min(n, c["ring"] or n, L - s) for L, n, s in zip(lens, counts, starts))
        read = sum(L - s for L, s in zip(lens, starts))
        return dict(bytes=hkv * (new * (4 * D + token) + (read - fresh) * token + read * 4 * D) + 12 * len(lens), flops=4 * D * hkv * new + 2 * D * hkv * read)
    total = flops = 0.0
    for L, n in zip(lens, counts):
        w = c["window"] or L
        keys = min(L, w + n - 1)
        pairs = sum(min(L - n + t + 1, w) for t in range(n))
        total += hkv * ((keys - n) * token + n * (4 * D + token)) + n * c["hq"] * 4 * D + 4 * (keys // PAGE) + 8
        flops += 4 * D * c["hq"] * pairs
    return dict(bytes=total + 4 * c["hq"], flops=flops)


# ---------------------------------------------------------------- the definition in 64 bits
def _grid():
    """The finite e4m3 values of no sign, ascending: 2^-9 m below 2^-6, then 2^(e-7) (1 + m / 8) up to 448."""
    return torch.tensor([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127], dtype=torch.float64, device="cuda")


def _stored(x):
    """The value on e4m3's grid and the scale of each element and row of x."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, (top / 448).float().double(), torch.ones_like(top))
    y = (x / scale).float().double()
    grid = _grid()
    # the index of the nearest value: equal distances to the even one
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(y.abs(), mid), torch.bucketize(y.abs(), mid, right=True)
    at = torch.where((low != high) & (low % 2 == 1), high, low)
    return torch.sign(y) * grid[at], scale[..., 0]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rotate":
        outs = dict(v=s["v"].double())
        axis = _sections(c)[1]
        for x in "qk":
            y = s[x].double()
            if c["norm"]:
                y = y / ((y ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * s[x + "_weight"].double()
            z = torch.empty_like(y)
            for i in range(HALF):
                at = s["positions"][axis[i]].long()
                co, si = s["rope_cos"][at, i].double()[:, None], s["rope_sin"][at, i].double()[:, None]
                z[..., i] = y[..., i] * co - y[..., i + HALF] * si
                z[..., i + HALF] = y[..., i + HALF] * co + y[..., i] * si
            outs[x] = z
        return dict(q=outs["q"], k=outs["k"], v=outs["v"])
    lens = _lens(c)
    counts = _counts(c, lens)
    H, W = c["hkv"], c.get("ring", 0)
    if c["op"] == "attend" and sum(lens) * max(counts) * c["hq"] > 2 ** 34:
        return None
    codes, scales = (x.clone() for x in _cache(s).values())
    flat_c, flat_s = codes.view(torch.uint8).view(-1, 2 * PAGE * D), scales.view(-1, 2 * PAGE)
    vals = flat_c.view(torch.float8_e4m3fn).double()

    def where(b, cells):
        """Blocks [cells, H] and slots of positions of sequence b."""
        if W:
            return (b * H + torch.arange(H, device="cuda")) * (W // PAGE) + (cells % W // PAGE)[:, None], cells % PAGE
        return s["block_table"][b].long()[cells // PAGE][:, None] * H + torch.arange(H, device="cuda"), cells % PAGE

    d = torch.arange(D, device="cuda")
    for b, (L, n) in enumerate(zip(lens, counts)):
        m = min(n, W) if W else n
        if m == 0:
            continue
        blk, slot = where(b, torch.arange(L - m, L, device="cuda"))
        for half, new in enumerate((s["k_new"], s["v_new"])):
            y, sc = _stored(new[b, n - m : n])
            at = slot[:, None, None] * D + d if half == 0 else PAGE * D + d * PAGE + slot[:, None, None]
            vals[blk[..., None], at] = y
            flat_s[blk, half * PAGE + slot[:, None]] = sc.float()

    def rows(b, cells):
        blk, slot = where(b, cells)
        k = vals[blk[..., None], slot[:, None, None] * D + d] * flat_s[blk, slot[:, None]].double()[..., None]
        v = vals[blk[..., None], PAGE * D + d * PAGE + slot[:, None, None]] * flat_s[blk, PAGE + slot[:, None]].double()[..., None]
        return k, v

    state = dict(codes=vals.view(codes.shape), scales=scales)
    if c["op"] == "store":
        starts, _ = _back(c, lens, counts)
        k_out, v_out = torch.zeros_like(s["k_out"], dtype=torch.float64), torch.zeros_like(s["v_out"], dtype=torch.float64)
        for b, (L, st) in enumerate(zip(lens, starts)):
            if L > st:
                k_out[b, : L - st], v_out[b, : L - st] = rows(b, torch.arange(st, L, device="cuda"))
        return dict(state, k=k_out, v=v_out)
    G = c["hq"] // H
    q = s["q"].view(c["batch"], c["tokens"], H, G, D)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(lens, counts)):
        if not n:
            continue
        cell = torch.arange(L, device="cuda")
        k, v = rows(b, cell)
        at = torch.arange(L - n, L, device="cuda")[:, None]
        see = cell <= at
        if c["window"]:
            see &= cell > at - c["window"]
        for h in range(H):
            x = torch.einsum("tgd,jd->tgj", q[b, :n, h].double(), k[:, h]) * SCALE
            x.masked_fill_(~see[:, None, :], -math.inf)
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"].double().view(H, G)[h][None, :, None].expand(n, G, 1)], -1)
            out[b, :n, h] = torch.einsum("tgj,jd->tgd", torch.softmax(x, -1)[..., :L], v[:, h])
    return dict(state, out=out.view(s["q"].shape))
