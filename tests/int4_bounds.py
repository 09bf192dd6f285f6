"""What attention over the 4-bit cache may differ by from 64 bits, row by row, and data on
which a token lost or added shows. Written from the kernels' roundings; all in numpy.

u = 2^-8 is half a step of bf16, relative; a rounding is off by at most u |x|, and by at most
u |x| / sqrt(3) in the root mean square (x anywhere in a binade: the step is that of its
start)."""
import numpy as np

import int4_ref as ref

U = 2.0 ** -8
FEW_ROWS = 32   # rows of a KV head (tokens times query heads) that the kernel for few takes


def params(cache, layer, slots):
    """((codes, s, lo) of K, the same of V) of slots: float64 [tokens, heads, D], [.., groups]."""
    D, g = cache.dim, cache.dim // cache.group
    slots = np.asarray(slots, dtype=np.int64)
    rows = cache.data[layer][slots // cache.page, :, slots % cache.page // 16]
    tok = slots % 16
    kv = cache.values(layer, slots)[:2]
    out = []
    for x, base in zip(kv, (8 * D, 16 * D + 64 * g)):
        at = (base + tok[:, None] * 4 * g + np.arange(4 * g))[:, None]
        raw = np.take_along_axis(rows, np.broadcast_to(at, rows.shape[:2] + (4 * g,)), 2)
        w = np.ascontiguousarray(raw).view(np.uint16).reshape(rows.shape[:2] + (g, 2))
        s, lo = (ref.from_bits(w[..., i]).astype(np.float64) for i in range(2))
        of = np.arange(D) // cache.group
        safe = np.where(s > 0, s, 1)
        out.append((np.rint((x - lo[..., of]) / safe[..., of]), s, lo))
    return out


def attention(cache, layer, q, cu, lens, table, window, sinks, scale, lose=()):
    """(o, most, mean): float64 [tokens, q_heads, D], rows of requests without any token 0.

    `most` bounds |out - o| for requests with few rows (inf for the others, of which only the
    mean is bounded): u |o| (the result), u sum p s |n - 8| (p s to bf16, before it meets n -
    8), 2 d sum p |v| for scores off by d (the sum of a group's q in two bf16 parts, 2^-16, and
    fp32 sums, 2^-20 of sum |scale q k|), and fp32 sums: 2^-23 a step of 16 tokens.
    `mean` is the mean square of the error that independent roundings give at the most. Few:
    u^2 / 3 (o^2 + sum (p s (n - 8))^2). Many: u^2 / 3 (o^2 + 2 sum (p v)^2 (p and v^ to bf16) +
    sum (p (v - o))^2 scale^2 sum (q k)^2 (k^ to bf16 moves a score, and the p's sum to 1)).
    `lose`: tokens that this oracle leaves out, to see what the bounds notice."""
    T, qh, D = q.shape
    heads = cache.shape[3]
    ratio = qh // heads
    of = np.arange(D) // cache.group
    o, most, mean = (np.zeros(q.shape) for _ in range(3))
    q = q.astype(np.float64)
    for r in range(len(lens)):
        a, b, m = int(cu[r]), int(cu[r + 1]), int(lens[r])
        few = (b - a) * ratio <= FEW_ROWS
        if a == b:
            continue
        if not few:
            most[a:b] = np.inf
        if m == 0:
            continue
        j = np.arange(m)
        x = m - (b - a) + np.arange(b - a)
        vis = j[None] <= x[:, None]
        if window:
            vis &= (x[:, None] - j[None] < window) | (j[None] < sinks)
        used = np.nonzero(vis.any(0))[0]
        if not len(used):
            continue
        slots = table[r][used // cache.page].astype(np.int64) * cache.page + used % cache.page
        vis = vis[:, used] & ~np.isin(used, lose)[None]
        rows = vis.any(1)
        (kn, ks, kl), (vn, vs, vl) = params(cache, layer, slots)
        for h in range(heads):
            k = kl[:, h][:, of] + ks[:, h][:, of] * kn[:, h]
            v = vl[:, h][:, of] + vs[:, h][:, of] * vn[:, h]
            w = vs[:, h][:, of] * (vn[:, h] - 8)
            top = (np.abs(kl[:, h]) + 15 * ks[:, h])[:, of]
            for e in range(h * ratio, (h + 1) * ratio):
                y = q[a:b, e]
                z = np.where(vis, y @ k.T * scale, -np.inf)
                p = np.exp(z - np.where(rows, z.max(1), 0)[:, None])
                p /= np.where(rows, p.sum(1), 1)[:, None]
                out = p @ v
                mass, steps = p @ np.abs(v), p @ np.abs(w)
                sums = (vis.sum(1)[:, None] / 16 + 64) * 2.0 ** -23 * (mass + 2 * steps)
                if few:
                    group = np.abs(y.reshape(len(y), -1, cache.group).sum(2)) @ np.abs(kl[:, h]).T
                    d = (np.where(vis, 2.0 ** -16 * group + 2.0 ** -20 * np.abs(y) @ top.T, 0) * abs(scale)).max(1)
                    fixed = np.expm1(2 * d)[:, None] * mass + sums
                    most[a:b, e] = U * np.abs(out) + U * steps + fixed
                    mean[a:b, e] = U ** 2 / 3 * (out ** 2 + p ** 2 @ w ** 2) + fixed ** 2
                else:
                    d = np.where(vis, 2.0 ** -20 * np.abs(y) @ np.abs(k).T, 0).max(1) * abs(scale)
                    moved = p ** 2 * (y ** 2 @ (k ** 2).T) * scale ** 2
                    # sum moved (v - o)^2, multiplied out
                    spread = moved @ v ** 2 - 2 * out * (moved @ v) + out ** 2 * moved.sum(1)[:, None]
                    fixed = np.expm1(2 * d)[:, None] * mass + sums
                    mean[a:b, e] = U ** 2 / 3 * (out ** 2 + 2 * p ** 2 @ v ** 2 + spread) + fixed ** 2
                o[a:b, e] = out
    return o, most, mean


# The mean square over a call, of 2^13 values and more, against the mean of `mean`: the bound
# takes every step at a binade's start; with mantissas spread over it the root is 0.74 of
# that (sqrt of (1 - 1/4) / (2 ln 2)), which leaves 1.5 to 1.1 for chance.
ROOM = 1.1


def check(out, o, most, mean):
    err = np.abs(out.astype(np.float64) - o)
    assert np.isfinite(err).all()
    over = err - most
    assert (over <= 0).all(), (float(over.max()), np.unravel_index(over.argmax(), over.shape))
    got, may = np.sqrt((err ** 2).mean()), np.sqrt(mean.mean())
    assert got <= ROOM * may, (got, may)


def whole_numbers(rng, *shape, group):
    """V values -8 .. 7 whose groups have lo = -8 and s = 1: exact in every form."""
    v = rng.integers(-8, 8, shape).astype(np.float32).reshape(shape[:-1] + (-1, group))
    v[..., 0], v[..., 1] = -8, 7
    return v.reshape(shape)


def counted(cache, layer, cu, lens, table, window, sinks, heads, ratio, lose=()):
    """(o, bound) where every visible token has the same weight and V holds whole_numbers: the
    mean of whole numbers. Weights are powers of two and all sums exact, so what is left is
    the quotient (2^-22) and the result's rounding."""
    T, D = int(cu[-1]), cache.dim
    o = np.zeros((T, heads * ratio, D))
    for r in range(len(lens)):
        a, b, m = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if a == b or m == 0:
            continue
        j = np.arange(m)
        reach = table[r][j // cache.page] >= 0
        slots = np.where(reach, table[r][j // cache.page], 0).astype(np.int64) * cache.page + j % cache.page
        v = cache.values(layer, slots)[1]
        x = m - (b - a) + np.arange(b - a)
        vis = j[None] <= x[:, None]
        if window:
            vis &= (x[:, None] - j[None] < window) | (j[None] < sinks)
        assert reach[vis.any(0)].all()
        vis &= ~np.isin(j, lose)[None]
        n = np.maximum(vis.sum(1), 1)
        mean = np.einsum("xj,jhd->xhd", vis.astype(np.float64), v) / n[:, None, None]
        o[a:b] = np.repeat(mean, ratio, axis=1)
    return o, (U + 2.0 ** -21) * np.abs(o) + 2.0 ** -126
