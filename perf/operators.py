"""The operators that keep a paged KV cache at a bounded size, as measured cases.

  decode  one new token per sequence: append, attention over the paged cache (bf16 or fp8 blocks), and every
          attended token's attention weight (summed over the query heads of its KV head) added to its cell
  prompt  the same for several new tokens per sequence (causal): draft verification, prompt chunks
  evict   every sequence longer than `keep` shrunk to `keep` cells per KV head: the first and the last cells
          stay, and of the cells between them those of the largest accumulated weight

Layouts are the framework's: pools [pages, Hkv, 16, 64] (fp8: [pages, Hkv, 2176] blocks), weights
[pages, Hkv, 16] fp32, block tables [B, max pages], lengths counted after the append (0 = inactive slot).
"""
import math
import random

import torch

own = False

PAGE, D = 16, 64
SCALE = 0.125


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's stream at a common context: every layer waits for it, latency counts
        dict(name="decode_b1", op="decode", kv="bf16", batch=1, hq=64, hkv=8, lens="fixed", lo=4096, hi=4096, inactive=0, window=0, sinks=True),
        # the framework's batch-64 decode step
        dict(name="decode_b64", op="decode", kv="bf16", batch=64, hq=64, hkv=8, lens="uniform", lo=1024, hi=8192, inactive=0, window=0, sinks=True),
        # one very long sequence: split over the whole GPU and joined
        dict(name="decode_long1", op="decode", kv="bf16", batch=1, hq=64, hkv=8, lens="fixed", lo=131072, hi=131072, inactive=0, window=0, sinks=True),
        # the batch-64 step on the fp8 cache
        dict(name="decode_fp8_b64", op="decode", kv="fp8", batch=64, hq=64, hkv=8, lens="uniform", lo=1024, hi=8192, inactive=0, window=0, sinks=True),
        # serving slots of very different lengths, a quarter of them inactive, 16 query heads per KV head, a window that starts inside a page
        dict(name="decode_slots_window", op="decode", kv="bf16", batch=96, hq=64, hkv=4, lens="lognormal", lo=1, hi=16384, inactive=24, window=4001, sinks=False),
        # draft verification: up to four new tokens per sequence
        dict(name="prompt_verify", op="prompt", kv="bf16", batch=32, hq=64, hkv=8, lens="uniform", lo=1024, hi=8192, inactive=0, window=0, sinks=True, tokens=4, counts="ragged"),
        # the last tokens of a long prompt decide what is kept of it
        dict(name="prompt_observe", op="prompt", kv="bf16", batch=1, hq=64, hkv=8, lens="fixed", lo=131072, hi=131072, inactive=0, window=0, sinks=True, tokens=32, counts="full"),
        # a chunk of a prompt behind its history
        dict(name="prompt_chunk", op="prompt", kv="bf16", batch=1, hq=64, hkv=8, lens="fixed", lo=8192, hi=8192, inactive=0, window=0, sinks=True, tokens=512, counts="full"),
        # whole prompts of several users, of different lengths
        dict(name="prompt_fresh", op="prompt", kv="bf16", batch=4, hq=64, hkv=8, lens="uniform", lo=1201, hi=2048, inactive=0, window=0, sinks=True, tokens=2048, counts="whole"),
        # a cache that grew by 64 tokens brought back to its size
        dict(name="evict_step", op="evict", kv="bf16", batch=8, hq=64, hkv=8, lens="fixed", lo=4160, hi=4160, inactive=0, keep=4096, first=4, last=256),
        # a batch's prompts cut down before decoding (some are short enough already)
        dict(name="evict_b64", op="evict", kv="bf16", batch=64, hq=64, hkv=8, lens="uniform", lo=1000, hi=8192, inactive=0, keep=1024, first=4, last=129),
        # one long fp8 cache cut down
        dict(name="evict_fp8_long1", op="evict", kv="fp8", batch=1, hq=64, hkv=8, lens="fixed", lo=131072, hi=131072, inactive=0, keep=8192, first=4, last=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "evict"])
    g = rng.choice([1, 2, 4, 8, 8, 16])
    hkv = rng.choice([1, 2, 4, 8, 8, 12])
    c = dict(op=op, kv=rng.choice(["bf16", "bf16", "fp8"]) if op != "prompt" else "bf16", hq=g * hkv, hkv=hkv)
    if op == "prompt":
        t = _log_int(rng, 2, 1024)
        pairs = 2 ** 28 // max(64, g * hkv)  # (new token, position) pairs over the batch at most
        hi = max(t + 1, _log_int(rng, 64, max(128, min(65536, pairs // t))))
        b = max(1, min(_log_int(rng, 1, 48), pairs // (t * hi), 2 ** 18 // hi))
        c.update(batch=b, lens=rng.choice(["fixed", "uniform"]), lo=max(t, hi // 5), hi=hi, inactive=rng.choice([0, 0, b // 4]),
                 window=rng.choice([0, 0, _log_int(rng, 1, hi)]), sinks=rng.random() < 0.7, tokens=t, counts=rng.choice(["full", "ragged"]))
        return c
    hi = _log_int(rng, 3, 65536)
    b = max(1, min(_log_int(rng, 1, 128), 2 ** 18 // hi))
    c.update(batch=b, lens=rng.choice(["fixed", "uniform", "lognormal"]), lo=max(1, hi // 7), hi=hi, inactive=rng.choice([0, 0, b // 4]))
    if op == "decode":
        c.update(window=rng.choice([0, 0, 0, _log_int(rng, 1, hi)]), sinks=rng.random() < 0.7)
    else:
        keep = _log_int(rng, 1, max(2, hi - 1))
        last = rng.randint(0, keep // 2)
        c.update(keep=keep, first=rng.randint(0, min(8, keep - last)), last=last)
    return c


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
    """New tokens per sequence of a prompt case."""
    rng = random.Random("%d %s" % (c["tokens"], c["counts"]))
    if c["counts"] == "whole":
        return [min(L, c["tokens"]) for L in lens]
    if c["counts"] == "full":
        return [min(L, c["tokens"]) for L in lens]
    return [min(L, rng.randint(1, c["tokens"])) for L in lens]


# ---------------------------------------------------------------- inputs
class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=torch.float32)

    def blocks(self, *lead):
        """fp8 blocks: finite e4m3 codes of both signs, and scales of rows whose largest value is 2 to 3."""
        codes = torch.randint(0, 256, lead + (2 * PAGE * D,), generator=self.g, device="cuda", dtype=torch.uint8)
        codes = torch.where((codes & 127) == 127, codes - 1, codes)
        scales = (2 + self.uniform(*lead, 2 * PAGE)) / 448
        return torch.cat([codes, scales.view(torch.uint8)], -1).contiguous()


def prepare(case, seed):
    c, r = case, _Draw(seed)
    lens = _lens(c)
    B, hkv = c["batch"], c["hkv"]
    need = [-(-L // PAGE) for L in lens]
    pages = max(1, sum(need) + sum(need) // 10)
    cols = max(1, max(need))
    perm = torch.randperm(pages, generator=r.g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    at = torch.arange(cols, device="cuda")[None, :]
    bt = torch.where(at < n[:, None], perm[((n.cumsum(0) - n)[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32)
    s = dict(case=c, block_table=bt.contiguous(), seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if c["kv"] == "fp8":
        s["kv_cache"] = r.blocks(pages, hkv)
    else:
        s["k_cache"], s["v_cache"] = r.normal(pages, hkv, PAGE, D), r.normal(pages, hkv, PAGE, D)
    # accumulated weights: heavy-tailed, most tokens attended little
    w = -torch.log(r.uniform(pages, hkv, PAGE).clamp(min=1e-7)) ** 3 * -0.01
    s["weights"] = w.contiguous()
    if c["op"] == "evict":
        s["fresh"] = w.clone()
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((B, hkv, c["keep"]), dtype=torch.int32, device="cuda")
        return s
    lead = (B,) if c["op"] == "decode" else (B, c["tokens"])
    s["q"], s["k_new"], s["v_new"] = r.normal(*lead, c["hq"], D), r.normal(*lead, hkv, D), r.normal(*lead, hkv, D)
    s["sinks"] = r.normal(c["hq"]).float() if c["sinks"] else None
    s["out"] = torch.empty_like(s["q"])
    if c["op"] == "prompt":
        s["q_lens"] = torch.tensor(_counts(c, lens), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms
def _rows(cache, bt):
    """[B, Hkv, cells, D] in 32 bits of a bf16 pool."""
    x = cache[bt.clamp(min=0).long()].float()
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, D)


def _split(kv):
    """Views of fp8 blocks: K codes [.., 16, 64], V codes [.., 64, 16], K scales, V scales [.., 16]."""
    n = PAGE * D
    codes = kv[..., : 2 * n].view(torch.float8_e4m3fn)
    scales = kv[..., 2 * n :].view(torch.float32)
    return codes[..., :n].unflatten(-1, (PAGE, D)), codes[..., n:].unflatten(-1, (D, PAGE)), scales[..., :PAGE], scales[..., PAGE:]


def _rows_fp8(kv, bt):
    x = kv[bt.clamp(min=0).long()]
    k, v, ks, vs = _split(x)
    k = k.float() * ks[..., None]
    v = v.float().transpose(-1, -2) * vs[..., None]
    return [y.permute(0, 2, 1, 3, 4).reshape(y.shape[0], y.shape[2], -1, D) for y in (k, v)]


def _quantise(x):
    """e4m3 codes (as bytes) and the scale of each row."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / 448, torch.ones_like(top))
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale[..., 0]


def _append(s, pages, slots, at):
    """The new tokens [N, Hkv, D] at `at` into cells (pages[N], slots[N])."""
    k, v = s["k_new"][at], s["v_new"][at]
    if "kv_cache" not in s:
        s["k_cache"][pages, :, slots] = k
        s["v_cache"][pages, :, slots] = v
        return
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    kv, d = s["kv_cache"], torch.arange(D, device="cuda")
    heads = torch.arange(kv.shape[1], device="cuda")
    pg, sl, hd = pages[:, None, None], slots[:, None, None], heads[None, :, None]
    kv[pg, hd, sl * D + d] = kc
    kv[pg, hd, PAGE * D + d * PAGE + sl] = vc
    scales = kv.view(torch.float32)[..., 2 * PAGE * D // 4 :]
    scales[pages[:, None], heads, slots[:, None]] = ks
    scales[pages[:, None], heads, PAGE + slots[:, None]] = vs


def _plain_attention(s):
    c, bt = s["case"], s["block_table"]
    T = c.get("tokens", 1)
    q = s["q"].view(c["batch"], T, c["hkv"], -1, D)
    B, _, H, G, _ = q.shape
    L = s["seq_lens"].long()
    n = s["q_lens"].long() if "q_lens" in s else (L > 0).long()
    base = L - n
    t = torch.arange(T, device="cuda")
    j = torch.arange(bt.shape[1] * PAGE, device="cuda")
    # the new tokens first: every key is then read from the cache
    b_at, t_at = (t[None, :] < n[:, None]).nonzero(as_tuple=True)
    pos = base[b_at] + t_at
    pages = bt.long()[b_at, pos // PAGE]
    _append(s, pages, pos % PAGE, (b_at, t_at) if "q_lens" in s else b_at)
    k, v = (_rows(s["k_cache"], bt), _rows(s["v_cache"], bt)) if "kv_cache" not in s else _rows_fp8(s["kv_cache"], bt)
    p = (base[:, None] + t)[:, :, None]                                     # [B, T, 1] each query's position
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
    o = torch.matmul(x.view(B, H, T * G, -1), v).view(B, H, T, G, D).permute(0, 2, 1, 3, 4)
    s["out"].copy_(o.reshape(s["out"].shape))
    w = x.sum((2, 3)).transpose(1, 2)                                       # [B, cells, H]
    seen = see.any(1)
    b_at, j_at = seen.nonzero(as_tuple=True)
    pages, slots = bt.long()[b_at, j_at // PAGE], j_at % PAGE
    new = (j_at >= base[b_at])[:, None]
    s["weights"][pages, :, slots] = torch.where(new, w[b_at, j_at], s["weights"][pages, :, slots] + w[b_at, j_at])


def _move(s, b, h, src, dst):
    """Cell dst[N] <- cell src[N] of sequence b[N] and KV head h[N], all read before any is written."""
    bt = s["block_table"].long()
    ps, pd, ss, sd = bt[b, src // PAGE], bt[b, dst // PAGE], src % PAGE, dst % PAGE
    caches = [s["weights"]]
    if "kv_cache" in s:
        kv = s["kv_cache"]
        flat, d = kv.view(-1), torch.arange(D, device="cuda")
        f32 = kv.view(torch.float32).view(-1)
        blk_s, blk_d = (ps * kv.shape[1] + h) * kv.shape[2], (pd * kv.shape[1] + h) * kv.shape[2]
        at_s = torch.cat([(blk_s + ss * D)[:, None] + d, (blk_s + PAGE * D + ss)[:, None] + d * PAGE], 1)
        at_d = torch.cat([(blk_d + sd * D)[:, None] + d, (blk_d + PAGE * D + sd)[:, None] + d * PAGE], 1)
        two = torch.arange(2, device="cuda") * PAGE
        sc_s, sc_d = (blk_s // 4 + PAGE * D // 2 + ss)[:, None] + two, (blk_d // 4 + PAGE * D // 2 + sd)[:, None] + two
        codes, scales = flat[at_s], f32[sc_s]
        flat[at_d] = codes
        f32[sc_d] = scales
    else:
        caches += [s["k_cache"], s["v_cache"]]
    for x in caches:
        x[pd, h, sd] = x[ps, h, ss]


def _plain_evict(s):
    c, bt, L = s["case"], s["block_table"].long(), s["seq_lens"].long()
    keep, f, r = c["keep"], c["first"], c["last"]
    n = keep - f - r
    H = c["hkv"]
    cells = torch.arange(bt.shape[1] * PAGE, device="cuda")
    over = L > keep
    s["new_lens"].copy_(torch.minimum(L, torch.full_like(L, keep)))
    w = s["weights"][bt.clamp(min=0)].permute(0, 2, 1, 3).reshape(len(L), H, -1)
    middle = (cells >= f) & (cells[None, :] < (L - r)[:, None]) & over[:, None]
    w = torch.where(middle[:, None, :], w, torch.full_like(w, float("-inf")))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    stay = torch.zeros_like(w, dtype=torch.bool).scatter_(2, order[..., :n], True) & middle[:, None, :]
    low = cells < f + n
    hole = ~stay & low & (cells >= f) & over[:, None, None]
    more = stay & ~low
    idx = torch.arange(keep, device="cuda")
    kept = torch.where((idx[None, :] < L[:, None]) & (~over[:, None] | (idx < f + n)), idx, -1)
    kept = torch.where(over[:, None] & (idx >= f + n), (L - keep)[:, None] + idx, kept)
    kept = kept[:, None, :].repeat(1, H, 1)
    b, h, dst = hole.nonzero(as_tuple=True)       # both lists ascend within each (sequence, head)
    src = more.nonzero(as_tuple=True)[2]
    kept[b, h, dst] = src
    s["kept"].copy_(kept)
    b2, i2 = (over[:, None] & (idx >= f + n)).nonzero(as_tuple=True)
    b2, i2 = b2.repeat_interleave(H), i2.repeat_interleave(H)
    h2 = torch.arange(H, device="cuda").repeat(len(b2) // H)
    _move(s, torch.cat([b, b2]), torch.cat([h, h2]), torch.cat([src, i2 + (L[b2] - keep)]), torch.cat([dst, i2]))


def _caches(s):
    if "kv_cache" in s:
        n = 2 * PAGE * D
        return dict(codes=s["kv_cache"][..., :n].view(torch.float8_e4m3fn), scales=s["kv_cache"][..., n:].view(torch.float32))
    return dict(k=s["k_cache"], v=s["v_cache"])


def run(state):
    s, c = state, state["case"]
    if c["op"] == "evict":
        s["weights"].copy_(s["fresh"])  # the weights that the steps since the last eviction left
        if own:
            import paged_decode_attention_kv_gb300 as da
            if "kv_cache" in s:
                da.kv_evict_fp8(s["kv_cache"], s["weights"], s["block_table"], s["seq_lens"], s["new_lens"], s["kept"], c["first"], c["last"])
            else:
                da.kv_evict(s["k_cache"], s["v_cache"], s["weights"], s["block_table"], s["seq_lens"], s["new_lens"], s["kept"], c["first"], c["last"])
        else:
            _plain_evict(s)
        return dict(_caches(s), weights=s["weights"], new_lens=s["new_lens"], kept=s["kept"])
    if own:
        import paged_decode_attention_kv_gb300 as da
        if c["op"] == "prompt":
            da.decode_attn_paged_multi_weights(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["weights"], s["block_table"],
                                               s["seq_lens"], s["sinks"], c["window"], SCALE, s["out"], q_lens=s["q_lens"])
        elif "kv_cache" in s:
            da.decode_attn_paged_fp8_weights(s["q"], s["k_new"], s["v_new"], s["kv_cache"], s["weights"], s["block_table"], s["seq_lens"],
                                             s["sinks"], c["window"], SCALE, s["out"])
        else:
            da.decode_attn_paged_weights(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["weights"], s["block_table"],
                                         s["seq_lens"], s["sinks"], c["window"], SCALE, s["out"])
    else:
        _plain_attention(s)
    return dict(_caches(s), weights=s["weights"], out=s["out"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    lens = _lens(c)
    hq, hkv = c["hq"], c["hkv"]
    token = 4 * D if c["kv"] == "bf16" else 2 * D + 8  # bytes of K and V of one token and KV head
    if c["op"] == "evict":
        n = c["keep"] - c["first"] - c["last"]
        total = 0.0
        for L in lens:
            total += 8 + hkv * 4 * c["keep"]
            if L > c["keep"]:
                mid = L - c["first"] - c["last"]
                moved = n * (mid - n) / mid + c["last"]  # the weights do not depend on the position
                total += hkv * (4 * mid + 2 * moved * (token + 4)) + 4 * (L // PAGE)
        return dict(bytes=total + sum(8 * PAGE * hkv * -(-L // PAGE) for L in lens), flops=0.0)  # and the copy of the weights
    counts = _counts(c, lens) if c["op"] == "prompt" else [1 if L else 0 for L in lens]
    total = flops = 0.0
    for L, n in zip(lens, counts):
        w = c["window"] or L
        keys = min(L, w + n - 1)
        pairs = sum(min(L - n + t + 1, w) for t in range(n))
        total += hkv * ((keys - n) * token + 8 * (keys - n) + n * (4 * D + token + 4)) + n * hq * 4 * D + 4 * (keys // PAGE) + 4
        flops += 4 * D * hq * pairs
    return dict(bytes=total + 4 * hq, flops=flops)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    lens = _lens(c)
    H, G = c["hkv"], c["hq"] // c["hkv"]
    bt = s["block_table"].long()
    if c["op"] == "evict":
        keep, f, r = c["keep"], c["first"], c["last"]
        w = s["weights"]
        wout = w.clone()
        kept = torch.full((c["batch"], H, keep), -1, dtype=torch.int64, device="cuda")
        blank = dict.fromkeys(("codes", "scales") if "kv_cache" in s else ())
        pools = {} if blank else dict(k=s["k_cache"], v=s["v_cache"])
        outs = {k: v.clone() for k, v in pools.items()}
        for b, L in enumerate(lens):
            cell = torch.arange(L, device="cuda")
            pages, slots = bt[b, cell // PAGE], cell % PAGE
            if L <= keep:
                kept[b, :, :L] = cell
                continue
            vals = w[pages, :, slots].double()[f : L - r]                    # [middle, H]
            # the rank of each: how many are larger, or equal and earlier
            rank = torch.argsort(torch.argsort(-vals, dim=0, stable=True), dim=0, stable=True)
            for h in range(H):
                best = (rank[:, h] < keep - f - r).nonzero()[:, 0] + f
                stays = best[best < keep - r]
                comes = best[best >= keep - r]
                to = torch.arange(keep, device="cuda")
                free = torch.ones(keep, dtype=torch.bool, device="cuda")
                free[:f] = False
                free[keep - r :] = False
                free[stays] = False
                to[free.nonzero()[:, 0]] = comes
                to[keep - r :] = torch.arange(L - r, L, device="cuda")
                kept[b, h] = to
                wout[pages[:keep], h, slots[:keep]] = w[pages[to], h, slots[to]]
                for k, x in pools.items():
                    outs[k][pages[:keep], h, slots[:keep]] = x[pages[to], h, slots[to]]
        return dict(blank, **outs, weights=wout, new_lens=torch.tensor([min(L, keep) for L in lens], dtype=torch.int32), kept=kept.int())
    T = c.get("tokens", 1)
    counts = _counts(c, lens) if c["op"] == "prompt" else [1 if L else 0 for L in lens]
    q = s["q"].view(c["batch"], T, H, G, D)
    kn, vn = (x.view(c["batch"], T, H, D).double() for x in (s["k_new"], s["v_new"]))
    if c["kv"] == "fp8":
        def stored(x):
            x = x.float()
            top = x.abs().amax(-1, keepdim=True)
            scale = torch.where(top > 0, top / 448, torch.ones_like(top))
            return (x / scale).to(torch.float8_e4m3fn).double() * scale.double()
        kn, vn = stored(kn), stored(vn)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double()
    for b, (L, n) in enumerate(zip(lens, counts)):
        if not L:
            continue
        if sum(lens) * max(counts) * c["hq"] > 2 ** 34:
            return None
        cell = torch.arange(L, device="cuda")
        pages, slots = bt[b, cell // PAGE], cell % PAGE
        if c["kv"] == "fp8":
            k8, v8, ks, vs = _split(s["kv_cache"])
            blocks = bt[b, : -(-L // PAGE)]
            k = (k8[blocks].double() * ks[blocks].double()[..., None]).transpose(1, 2).reshape(-1, H, D)[:L]
            v = (v8[blocks].double() * vs[blocks].double()[..., None, :]).permute(0, 3, 1, 2).reshape(-1, H, D)[:L]
        else:
            k, v = s["k_cache"][pages, :, slots].double(), s["v_cache"][pages, :, slots].double()
        k[L - n :], v[L - n :] = kn[b, :n], vn[b, :n]
        at = torch.arange(L - n, L, device="cuda")[:, None]
        see = cell <= at
        if c["window"]:
            see &= cell > at - c["window"]
        for h in range(H):
            x = torch.einsum("tgd,jd->tgj", q[b, :n, h].double(), k[:, h]) * SCALE
            x.masked_fill_(~see[:, None, :], -math.inf)
            if s["sinks"] is not None:
                sink = s["sinks"].double().view(H, G)[h][None, :, None].expand(n, G, 1)
                x = torch.cat([x, sink], -1)
            x = torch.softmax(x, -1)[..., :L]
            out[b, :n, h] = torch.einsum("tgj,jd->tgd", x, v[:, h])
            mass = x.sum((0, 1))
            mass[: L - n] += weights[pages, h, slots][: L - n]
            seen = see.any(0)
            weights[pages[seen], h, slots[seen]] = mass[seen]
    caches = dict(codes=None, scales=None) if c["kv"] == "fp8" else dict(k=None, v=None)
    return dict(caches, weights=weights, out=out.view(s["q"].shape))
