"""Eviction from the 4-bit paged cache in plain numpy, for the tests, written from the
definitions in include/cachegen.h: attention weights of tokens in 64 bits, the choice of
tokens, their move within the cache's bytes, and the release of pages."""
import numpy as np

import int4_ref as ref


def _k_parts(cache, layer, slots):
    """s and mid = lo + 8 s of K's groups, spread over the channels: float64 [tokens, heads, D]."""
    D, g = cache.dim, cache.dim // cache.group
    slots = np.asarray(slots, dtype=np.int64)
    rows = cache.data[layer][slots // cache.page, :, slots % cache.page // 16]
    at = 8 * D + (slots % 16)[:, None] * 4 * g + np.arange(4 * g)
    par = np.take_along_axis(rows, np.broadcast_to(at[:, None], rows.shape[:2] + (4 * g,)), 2)
    par = ref.from_bits(par.copy().view(np.uint16)).reshape(rows.shape[:2] + (g, 2)).astype(np.float64)
    s, lo = par[..., 0], par[..., 1]
    return np.repeat(s, cache.group, -1), np.repeat(lo + 8 * s, cache.group, -1)


def weigh(cache, layer, q, cu, lens, table, window, sinks, scale, width):
    """The sums of attention weights and their bound, float64 [requests, heads, width]; NaN from a
    request's last token on. The bound: a score (in powers of two) is a sum in fp32, by groups, of
    products that are exact, its terms scale log2(e) |q| (8 s + |lo + 8 s|) at most in sum; some 30
    roundings of at most 2^-23 (a matrix instruction may cut where others round) of that sum move it
    by d, and 2^z by a factor within exp(+-2 d ln 2) (z and the row's sum). The exponentials have 2
    units in the last place, sums of up to 2^18 terms are kept in parts of 2^9 at most:
    together below 2^-12 of the weight itself."""
    T, qh, D = q.shape
    heads = cache.shape[3]
    ratio = qh // heads
    out = np.full((len(lens), heads, width), np.nan)
    tol = np.full(out.shape, np.nan)
    q = q.astype(np.float64)
    for r in range(len(lens)):
        a, b, m = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if m == 0:
            continue
        out[r, :, :m], tol[r, :, :m] = 0, 0
        j = np.arange(m)
        x = m - (b - a) + np.arange(b - a)
        vis = j[None, :] <= x[:, None]
        if window:
            vis &= (x[:, None] - j[None, :] < window) | (j[None, :] < sinks)
        used = np.nonzero(vis.any(0))[0]
        if not len(used):
            continue
        slots = table[r][used // cache.page].astype(np.int64) * cache.page + used % cache.page
        k, _, _ = cache.values(layer, slots)
        s, mid = _k_parts(cache, layer, slots)
        vis = vis[:, used]
        rows = vis.any(1)
        for h in range(qh):
            n = h // ratio
            z = np.where(vis, q[a:b, h] @ k[:, n].T * scale, -np.inf)
            size = np.where(vis, np.abs(q[a:b, h]) @ (8 * s[:, n] + np.abs(mid[:, n])).T * abs(scale), 0).max(1)
            with np.errstate(invalid="ignore"):
                p = np.exp(z - np.where(rows, z.max(1), 0)[:, None])
            p /= np.where(rows, p.sum(1), 1)[:, None]
            d = 30 * 2.0 ** -23 * size[:, None]
            out[r, n, used] += p.sum(0)
            tol[r, n, used] += (p * (np.expm1(2 * d) + 2.0 ** -12)).sum(0)
    return out, tol


def choose(weights, lens, budget, recent, sinks):
    """kept int32 [.., budget] and the new lengths."""
    kept = np.full(weights.shape[:-1] + (budget,), -1, np.int32)
    new = np.array(lens, dtype=np.int32).copy()
    for at in np.ndindex(*weights.shape[:-1]):
        m = int(lens[at[-2]])
        if m < 0 or m > weights.shape[-1]:
            continue
        if m <= budget:
            kept[at][:m] = np.arange(m)
            continue
        new[at[-2]] = budget
        first, last = np.arange(sinks), np.arange(m - recent, m)
        pick = budget - sinks - recent
        w = weights[at][sinks:m - recent].astype(np.float64)
        order = sorted(range(len(w)), key=lambda i: (np.isnan(w[i]), -w[i] if not np.isnan(w[i]) else 0, i))[:pick]
        kept[at] = np.concatenate([first, sinks + np.sort(np.array(order, dtype=np.int64)), last])
    return kept, new


def _token(cache, layer, head, slot):
    """Where a token of a head lies: its blob's bytes, and (offset, step 1 or the V pairs' halves) as index arrays."""
    D, g = cache.dim, cache.dim // cache.group
    page, tok = slot // cache.page, slot % 16
    blob = cache.data[layer, page, head, slot % cache.page // 16]
    pair = 8 * D + 64 * g + tok // 2 * D
    v = pair + np.arange(D).reshape(-1, 4)[:, 2 * (tok % 2):2 * (tok % 2) + 2].reshape(-1)
    at = np.concatenate([tok * (D // 2) + np.arange(D // 2), 8 * D + tok * 4 * g + np.arange(4 * g), v,
                         16 * D + 64 * g + tok * 4 * g + np.arange(4 * g)])
    return blob, at


def compact(cache, first_layer, kept, new_lens, lens, table, weights=None):
    """The cache's bytes (and weights) after the move, in place; kept [layers, requests, heads, budget]."""
    for l, r, h in np.ndindex(*kept.shape[:3]):
        n, m = int(new_lens[r]), int(lens[r])
        if n == m:
            continue
        src = [int(j) for j in kept[l, r, h, :n]]
        got = []
        for j in src:
            blob, at = _token(cache, first_layer + l, h, int(table[r][j // cache.page]) * cache.page + j % cache.page)
            got.append(blob[at].copy())
        for i, x in enumerate(got):
            blob, at = _token(cache, first_layer + l, h, int(table[r][i // cache.page]) * cache.page + i % cache.page)
            blob[at] = x
        if weights is not None:
            w = weights[l, r, h, src].copy()
            weights[l, r, h, :m] = 0
            weights[l, r, h, :n] = w


def release(table, lens, new_lens, free, nfree, page):
    """(table, free pages, their number, cu) after the call."""
    table, free, cu = table.copy(), free.copy(), [0]
    for r in range(len(lens)):
        a, b = -(-int(new_lens[r]) // page), -(-int(lens[r]) // page)
        free[nfree + cu[-1]:nfree + cu[-1] + b - a] = table[r, a:b]
        table[r, a:b] = -1
        cu.append(cu[-1] + b - a)
    return table, free, nfree + cu[-1], np.array(cu, np.int32)
