"""Plain 64-bit forms of the calls that accumulate attention weights and of the eviction, on
numpy arrays, for the tests: the definitions written out, one sequence and KV head at a time."""
import numpy as np


def step(q, keys, values, L, n, sinks, window, scale):
    """One sequence: q [T, Hq, D], keys / values [L, Hkv, D] after the append, n new tokens.
    Returns out [T, Hq, D], mass [L, Hkv] and seen [L] (float64, bool)."""
    T, Hq, D = q.shape
    Hkv = keys.shape[1]
    G = Hq // Hkv
    out, mass, seen = np.zeros((T, Hq, D)), np.zeros((L, Hkv)), np.zeros(L, bool)
    j = np.arange(L)
    for t in range(n):
        p = L - n + t
        see = (j <= p) & ((j > p - window) if window else True)
        seen |= see
        for g in range(Hkv):
            s = scale * q[t, g * G:(g + 1) * G] @ keys[see, g].T                 # [G, keys]
            top = s.max(1)
            if sinks is not None:
                top = np.maximum(top, sinks[g * G:(g + 1) * G])
            e = np.exp(s - top[:, None])
            den = e.sum(1)
            if sinks is not None:
                den = den + np.exp(sinks[g * G:(g + 1) * G] - top)
            P = e / den[:, None]
            out[t, g * G:(g + 1) * G] = P @ values[see, g]
            mass[see, g] += P.sum(0)
    return out, mass, seen


def weights_tolerance(q, keys, rows, L, scale):
    """Relative bound of an accumulated weight of one call. A score is a sum of 64 exact products
    of magnitude sum A (log2 units), each addition off by 2^-24 of a partial sum of at most A, and
    so is the row's log2 denominator, so 2^(s - lse) is off by ln 2 * 2 * 66 * A * 2^-24; the
    hardware exponentials add 2^-22 a piece, the denominator's longest chain of additions
    (L / 8 keys of one lane) and the weight's (rows) 2^-24 each; 64 more for the merges."""
    if L == 0:
        return 0.0
    D = q.shape[-1]
    A = np.abs(q).reshape(-1, D).max(0) @ np.abs(keys).reshape(-1, D).max(0) * scale * 1.4427
    return 2.0 ** -24 * (0.6932 * 132 * A + rows + L / 8 + 64)


def kept_cells(weights, L, keep, first, last):
    """kept[0..keep-1] of one sequence and KV head from its weights [L] (float32)."""
    if L <= keep:
        return np.concatenate([np.arange(L), np.full(keep - L, -1)]).astype(np.int64)
    n = keep - first - last
    mid = np.arange(first, L - last)
    w = weights[mid].astype(np.float64)
    rank = sorted(range(len(mid)), key=lambda i: (np.isnan(w[i]), 0.0 if np.isnan(w[i]) else -w[i], i))
    stay = np.zeros(L, bool)
    stay[mid[rank[:n]]] = True
    out = np.arange(keep)
    out[keep - last:] = np.arange(L - last, L)
    holes = [c for c in range(first, first + n) if not stay[c]]
    out[holes] = [c for c in range(first + n, L - last) if stay[c]]
    return out


def evict_maps(weights, block_table, lens, keep, first, last):
    """kept [B, Hkv, keep] and new_lens [B] from paged weights [pages, Hkv, 16]."""
    B, Hkv = len(lens), weights.shape[1]
    kept = np.zeros((B, Hkv, keep), np.int32)
    for b, L in enumerate(lens):
        c = np.arange(L)
        for g in range(Hkv):
            page = block_table[b, c // 16]
            ok = (page >= 0) & (page < weights.shape[0])
            w = np.where(ok, weights[np.where(ok, page, 0), g, c % 16], np.nan)
            kept[b, g] = kept_cells(w, int(L), keep, first, last)
    return kept, np.minimum(lens, keep).astype(np.int32)


def move(pool, block_table, lens, kept):
    """pool [pages, Hkv, 16, ...] after the moves kept says, out of place; a move into or out of a
    page outside the pool is skipped."""
    out = pool.copy()
    keep = kept.shape[2]
    for b, L in enumerate(lens):
        if L <= keep:
            continue
        dst = np.arange(keep)
        for g in range(kept.shape[1]):
            src = kept[b, g]
            ps, pd = block_table[b, src // 16], block_table[b, dst // 16]
            ok = (ps >= 0) & (ps < pool.shape[0]) & (pd >= 0) & (pd < pool.shape[0])
            out[pd[ok], g, dst[ok] % 16] = pool[ps[ok], g, src[ok] % 16]
    return out
