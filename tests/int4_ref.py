"""The 4-bit paged cache and its attention in plain numpy, for the tests:
written from the definitions in include/cachegen.h, one channel's place at a
time, values and attention in 64 bits."""
import numpy as np

EPS = 2.0 ** -8   # half a step of bf16, relative


def bf16_round(x):
    """fp32 -> the nearest bf16 value (ties to even), as fp32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return r.view(np.float32)


def bits(x):
    """bf16 bit patterns of fp32 values that are bf16."""
    return (np.ascontiguousarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def from_bits(b):
    return (np.asarray(b).astype(np.uint32) << 16).view(np.float32)


def quantise(x, group):
    """x fp32 (bf16 values) [..., D] -> codes uint8 [..., D], s and lo fp32 [..., D / group]."""
    y = np.asarray(x, dtype=np.float32).reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    with np.errstate(all="ignore"):
        lo, hi = y.min(-1), y.max(-1)
        # the format multiplies by 1 / 15 in fp32 (and does not divide)
        s = bf16_round(((hi - lo).astype(np.float32) * (np.float32(1.0) / np.float32(15.0))).astype(np.float32))
        top = (lo.astype(np.float64) + 15.0 * s.astype(np.float64)).astype(np.float32)
        bad = ~np.isfinite(y).all(-1) | ~np.isfinite(s) | ~(top < 2.0 ** 128 - 2.0 ** 119)   # rounds to inf from there on
        s, lo = np.where(bad, np.float32(0), s), np.where(bad, np.float32(0), lo)
        d = (y - lo[..., None]).astype(np.float32)
        n = np.rint((d / s[..., None]).astype(np.float32))
        n = np.where(s[..., None] > 0, np.minimum(n, 15), 0).astype(np.uint8)
    return n.reshape(x.shape), s.astype(np.float32), lo.astype(np.float32)


class Cache:
    """Bytes of a cache as cg_int4_store writes them."""

    def __init__(self, layers, pages, page, heads, dim, group, fill=0):
        self.shape = (layers, pages, page, heads, dim, group)
        self.page, self.dim, self.group = page, dim, group
        self.blob = 16 * (dim + 8 * (dim // group))
        self.data = np.full((layers, pages, heads, page // 16, self.blob), fill, dtype=np.uint8)
        c = np.arange(dim)
        self.k_at = c % 32 // 8 * (dim // 8) + c // 32 * 4 + c % 8 // 2
        self.v_at = c % 32 // 4 * (dim // 8) + c // 32 * 4 + c % 4 // 2

    def store(self, layer, k, v, slots):
        """k, v fp32 [tokens, heads, D]."""
        D, g = self.dim, self.dim // self.group
        kn, ks, kl = quantise(k, self.group)
        vn, vs, vl = quantise(v, self.group)
        for t, slot in enumerate(np.asarray(slots).tolist()):
            if slot < 0:
                continue
            p, i = divmod(slot, self.page)
            rows = self.data[layer, p, :, i // 16]
            tok = i % 16
            for n, at in ((kn[t], tok * (D // 2) + self.k_at),
                          (vn[t], 8 * D + 64 * g + tok // 2 * D + tok % 2 * 2 + self.v_at)):
                rows[:, at[0::2]] = n[:, 0::2] | n[:, 1::2] << 4
            for s, lo, base in ((ks[t], kl[t], 8 * D), (vs[t], vl[t], 16 * D + 64 * g)):
                par = np.stack((bits(s), bits(lo)), -1).reshape(s.shape[0], -1)
                rows[:, base + tok * 4 * g:base + (tok + 1) * 4 * g] = par.view(np.uint8)

    def values(self, layer, slots):
        """(k, v, s of v) of slots, float64 [tokens, heads, D]."""
        D, g = self.dim, self.dim // self.group
        slots = np.asarray(slots, dtype=np.int64)
        rows = self.data[layer][slots // self.page, :, slots % self.page // 16]
        tok = (slots % 16)[:, None]
        of = np.arange(D) // self.group
        sh = (np.arange(D) % 2 * 4)[None, None, :]
        out = []
        for at, base in ((tok * (D // 2) + self.k_at, 8 * D),
                         (8 * D + 64 * g + tok // 2 * D + tok % 2 * 2 + self.v_at, 16 * D + 64 * g)):
            code = np.take_along_axis(rows, np.broadcast_to(at[:, None], rows.shape[:2] + (D,)), 2)
            code = (code >> sh) & 15
            word = (base + (tok * g + of) * 4)[:, None]
            b = [np.take_along_axis(rows, np.broadcast_to(word + i, rows.shape[:2] + (D,)), 2)
                 .astype(np.uint16) for i in range(4)]
            s = from_bits(b[0] | b[1] << 8).astype(np.float64)
            lo = from_bits(b[2] | b[3] << 8).astype(np.float64)
            out += [lo + s * code, s]
        return out[0], out[2], out[3]


def attention(cache, layer, q, cu, lens, table, window, sinks, scale):
    """out and its bound: float64 [tokens, q_heads, D]. The bound counts, per
    element and relative to what is summed: the rounding of the result to
    bf16 (EPS |o|); of the probabilities, or their products with s, to bf16
    and of v^ to bf16 (EPS of sum p |v^| each, and EPS of sum p 8 s where s
    (n - 8) is summed apart from its offset); and of k^ to bf16, which moves a
    score by up to d = EPS scale sum |q k^|, hence every probability by a
    factor within exp(+-2 d). fp32 sums add less than 2^-14 of sum p (|v^| + 16 s)
    (16 bits of slack over 2^-24 for sums of up to 2^10 terms a thread)."""
    T, qh, D = q.shape
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    ratio = qh // cache.shape[3]
    q = q.astype(np.float64)
    for r in range(len(lens)):
        a, b, m = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if a == b or m == 0:
            continue
        j = np.arange(m)
        x = m - (b - a) + np.arange(b - a)
        vis = j[None, :] <= x[:, None]
        if window:
            vis &= (x[:, None] - j[None, :] < window) | (j[None, :] < sinks)
        used = np.nonzero(vis.any(0))[0]
        if not len(used):
            continue
        pages = table[r][used // cache.page].astype(np.int64)
        assert (pages >= 0).all()
        k, v, s = cache.values(layer, pages * cache.page + used % cache.page)
        vis = vis[:, used]
        rows = vis.any(1)
        for h in range(qh):
            kh, vh, sh = k[:, h // ratio], v[:, h // ratio], s[:, h // ratio]
            z = np.where(vis, q[a:b, h] @ kh.T * scale, -np.inf)
            d = np.where(vis, np.abs(q[a:b, h]) @ np.abs(kh).T * abs(scale) * EPS, 0).max(1)
            with np.errstate(invalid="ignore"):
                p = np.exp(z - np.where(rows, z.max(1), 0)[:, None])
            p /= np.where(rows, p.sum(1), 1)[:, None]
            o, mass = p @ vh, p @ np.abs(vh)
            steps = p @ (8 * sh)
            out[a:b, h] = o
            tol[a:b, h] = EPS * np.abs(o) + EPS * (2 * mass + steps) + \
                np.expm1(2 * d)[:, None] * mass + 2.0 ** -14 * (mass + 2 * steps)
    return out, tol
