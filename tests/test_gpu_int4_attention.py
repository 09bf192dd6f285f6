"""Attention over the 4-bit cache against tests/int4_bounds.py: that every visible token counts
once and no other does, wherever the kernels cut the tokens, and that the error is that of
the roundings that the kernels name."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_bounds as bounds  # noqa: E402
import int4_ref as ref  # noqa: E402
from kv_cache_compression_03_gb300 import cachegen as cg  # noqa: E402

from test_gpu_int4 import FORMATS, _batch, _copy, _dev, _filled, _ints, _np, _pair, _rand  # noqa: E402

# query tokens, cache tokens, query heads of a KV head: rows of one token, drafts of 16 and 32
# rows, one and two row tiles (33 .. 128, 256), prompts; lengths that one warp, one block and
# several blocks take, and that fill no blob, no tile and no page
SHAPES = [([1] * 9, [1, 15, 16, 17, 128, 129, 700, 3100, 9001], 4),
          ([1] * 3, [255, 2055, 5000], 7),
          ([4, 4, 2], [4, 1500, 9001], 4),
          ([8, 7], [2000, 4111], 4),
          ([9, 16], [300, 6007], 4),
          ([64, 33], [3100, 1025], 4),
          ([300, 1, 140], [300, 513, 900], 2),
          ([70] * 10, [70 + 130 * i for i in range(10)], 2)]
WINDOWS = [(0, 0), (1, 0), (129, 3), (700, 37)]


def _shape(i):
    return pytest.param(*SHAPES[i], id=str(i))


def _out(got, q, cu, nkv, table, **kw):
    out = got.attention(_dev(q), _ints(cu), _ints(nkv), _ints(table), **kw)
    got.check()
    return _np(out)


@pytest.mark.parametrize("nq,nkv,ratio", [_shape(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("dim,group,page", [(128, 32, 16), (64, 64, 48)])
def test_error_is_that_of_the_roundings(nq, nkv, ratio, window, sinks, dim, group, page):
    rng = np.random.default_rng(sum(nkv) + window)
    heads = 2
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = _rand(rng, int(cu[-1]), heads * ratio, dim)
    out = _out(got, q, cu, nkv, table, window=window, sinks=sinks)
    bounds.check(out, *bounds.attention(want, 0, q, cu, nkv, table, window, sinks, dim ** -0.5))


@pytest.mark.parametrize("dim,group", [f for f in FORMATS if f not in ((128, 32), (64, 64))])
@pytest.mark.parametrize("i", [0, 2, 5])
def test_error_of_the_other_formats(dim, group, i):
    test_error_is_that_of_the_roundings(*SHAPES[i], 0, 0, dim, group, 32)


@pytest.mark.parametrize("nq,nkv,ratio", [_shape(i) for i in range(len(SHAPES))] +
                         [([1, 2], [40000, 33333], 4), ([20], [30000], 4)])
@pytest.mark.parametrize("window,sinks", WINDOWS + [(16, 16), (5000, 130)])
def test_every_visible_token_counts_once(nq, nkv, ratio, window, sinks):
    """Equal weights and whole numbers in V: the result is a sum of exactly the visible tokens."""
    rng = np.random.default_rng(sum(nkv) + window)
    heads, page, dim, group = 2, 16, 64, 32
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _pair(1, pages, page, heads, dim, group, fill=0xFF)
    for r, m in enumerate(nkv):
        x = np.arange(m)
        k, v = _rand(rng, m, heads, dim), bounds.whole_numbers(rng, m, heads, dim, group=group)
        want.store(0, k, v, table[r][x // page] * page + x % page)
    _copy(want, got)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = np.zeros((int(cu[-1]), heads * ratio, dim), np.float32)
    for most in (None, max(nq)):
        out = _out(got, q, cu, nkv, table, window=window, sinks=sinks, max_q_len=most)
        o, tol = bounds.counted(want, 0, cu, nkv, table, window, sinks, heads, ratio)
        over = np.abs(out - o) - tol
        assert (over <= 0).all(), (float(over.max()), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("nq,nkv,ratio", [([1, 1], [3100, 700], 8), ([4, 3], [5000, 1600], 4), ([16, 16], [3100, 700], 4),
                                          ([64], [2200], 4), ([260], [900], 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 20)])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_query_finds_its_token(nq, nkv, ratio, window, sinks, dim):
    """K is signs, a query the sum of a visible token's and one that it must not see: the
    result is the visible one's V, for tokens at the borders of blobs, tiles, window and sinks."""
    rng = np.random.default_rng(sum(nkv) + window + dim)
    heads, page, group = 2, 32, 64
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _pair(1, pages, page, heads, dim, group, fill=0xFF)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q, o = np.zeros((int(cu[-1]), heads * ratio, dim), np.float32), np.zeros((int(cu[-1]), heads * ratio, dim))
    for r, m in enumerate(nkv):
        k = rng.choice([-1.0, 1.0], (m, heads, dim)).astype(np.float32)
        v = bounds.whole_numbers(rng, m, heads, dim, group=group)
        x = np.arange(m)
        want.store(0, k, v, table[r][x // page] * page + x % page)
        for i in range(nq[r]):
            at = m - nq[r] + i
            low = max(0, at + 1 - window) if window else 0
            seen = np.concatenate([np.arange(min(sinks, low)), np.arange(low, at + 1)])
            not_seen = np.setdiff1d(x, seen)
            edges = [low, low + 1, at, at - 1, 0, sinks - 1]
            edges += [t + d for t in rng.integers(0, m // 128 + 1, 3) * 128 for d in (-1, 0, 1)]
            edges += [t + d for t in rng.integers(0, m // 16 + 1, 3) * 16 for d in (-1, 0)]
            edges = [t for t in edges if t in seen]
            wrong = [t for t in (low - 1, sinks, at + 1, at + 2) if t in not_seen]
            for h in range(heads * ratio):
                t = edges[(h + i) % len(edges)] if (h + i) % 3 else int(rng.choice(seen))
                y = k[t, h // ratio].copy()
                if wrong:
                    y += k[wrong[(h + i) % len(wrong)], h // ratio]
                q[cu[r] + i, h], o[cu[r] + i, h] = y, v[t, h // ratio]
    _copy(want, got)
    scale = 4.0
    plain = ref.attention(want, 0, q, cu, nkv, table, window, sinks, scale)[0]
    clear = np.abs(plain - o).max(2) < 0.01       # (now and then two tokens are too much alike)
    assert clear.mean() > 0.97
    out = _out(got, q, cu, nkv, table, window=window, sinks=sinks, scale=scale)
    # p s, p and the result to bf16: 2^-8 of 8, three times
    assert np.abs(out - o)[clear].max() <= 3 * 8 * bounds.U + 0.01


@pytest.mark.parametrize("dim,group,ratio", [(128, 32, 4), (64, 64, 4), (128, 64, 16)])
@pytest.mark.parametrize("power", [96, 112, 122])
def test_large_values_of_v(dim, group, ratio, power):
    """Few rows: equal scores, so that the sum of p V passes fp32's range long before V does."""
    rng = np.random.default_rng(power)
    heads, page, nq, nkv = 2, 32, [1, 2, 1, 1], [256, 700, 9001, 70000]
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _pair(1, pages, page, heads, dim, group, fill=0xFF)
    for r, m in enumerate(nkv):
        x = np.arange(m)
        v = bounds.whole_numbers(rng, m, heads, dim, group=group) * np.float32(2.0 ** power)
        want.store(0, _rand(rng, m, heads, dim), v, table[r][x // page] * page + x % page)
    _copy(want, got)
    cu = np.concatenate([[0], np.cumsum(nq)])
    out = _out(got, np.zeros((5, heads * ratio, dim), np.float32), cu, nkv, table, max_q_len=2)
    o, tol = bounds.counted(want, 0, cu, nkv, table, 0, 0, heads, ratio)
    assert np.isfinite(out).all() and (np.abs(out - o) <= tol).all()


@pytest.mark.parametrize("dim,group,ratio", [(128, 32, 4), (64, 64, 16)])
def test_values_of_v_of_every_size_side_by_side(dim, group, ratio):
    """Stretches of tokens at 1, 2^20, 2^60 and 2^120: warps and parts come together with factors
    of their own. Under the window a request sees one or two of the sizes."""
    rng = np.random.default_rng(dim)
    heads, page, window = 1, 16, 700
    nq, nkv = [1] * 6, [900, 2000, 2900, 3900, 1300, 60]
    powers = [0, 20, 60, 120]
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _pair(1, pages, page, heads, dim, group, fill=0xFF)
    for r, m in enumerate(nkv):
        x = np.arange(m)
        v = _rand(rng, m, heads, dim) * np.exp2(np.array(powers)[x // 1000])[:, None, None]
        want.store(0, _rand(rng, m, heads, dim), ref.bf16_round(v.astype(np.float32)), table[r][x // page] * page + x % page)
    _copy(want, got)
    cu = np.arange(7)
    q = _rand(rng, 6, heads * ratio, dim)
    for w in (0, window):
        out = _out(got, q, cu, nkv, table, window=w, max_q_len=1)
        o, most, _ = bounds.attention(want, 0, q, cu, nkv, table, w, 0, dim ** -0.5)
        assert np.isfinite(out).all() and (np.abs(out - o) <= most).all()


# ordinary scores whose scale and whose products q.k are not
SCALES = [(0.0, 2.0 ** 60, 2.0 ** 58), (2.0 ** 70, 1.0, 2.0 ** -74), (-2.0 ** 100, 2.0 ** -54, 2.0 ** -50),
          (2.0 ** -100, 2.0 ** 30, 2.0 ** 67), (2.0 ** -126, 2.0 ** 22, 2.0 ** 101)]


def _scales(nq, ratio, scale, kscale, qscale):
    rng = np.random.default_rng(nq)
    nkv, page, heads, dim, group = [90, 700], 16, 2, 128, 32
    table, pages = _batch(rng, [nq] * 2, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group, scale=kscale)
    cu = [0, nq, 2 * nq]
    q = _rand(rng, 2 * nq, heads * ratio, dim, scale=qscale)
    out = _out(got, q, cu, nkv, table, scale=scale)
    bounds.check(out, *bounds.attention(want, 0, q, cu, nkv, table, 0, 0, scale))


@pytest.mark.parametrize("scale,kscale,qscale", SCALES)
def test_scales_of_every_size_many_rows(scale, kscale, qscale):
    _scales(90, 2, scale, kscale, qscale)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_a_scale_of_zero_keeps_what_is_not_finite(bad):
    q = torch.ones(80, 2, 64, dtype=torch.bfloat16, device="cuda")
    q[7, 1, 3] = bad
    cache = cg.Int4Cache(1, 10, 16, 1, 64, 64)
    cache.store(torch.ones(100, 1, 64, dtype=torch.bfloat16, device="cuda"),
                torch.ones(100, 1, 64, dtype=torch.bfloat16, device="cuda"), _ints(range(100)))
    for n in (80, 1):
        out = cache.attention(q[7:7 + n] if n == 1 else q, _ints([0, n]), _ints([100]), _ints([range(10)]), scale=0.0)
        at = 0 if n == 1 else 7
        assert torch.isnan(out[at, 1]).all() and bool((out[at, 0] == 1).all()) and not torch.isnan(out[at + 1:]).any()


@pytest.mark.parametrize("nq,ratio", [(1, 4), (3, 8)])
@pytest.mark.parametrize("scale,kscale,qscale", SCALES)
def test_scales_of_every_size_few_rows(scale, kscale, qscale, nq, ratio):
    _scales(nq, ratio, scale, kscale, qscale)


# 2^-149 is fp32's last bit; 2^-149 2^(133 - 90) a step of 16 tokens, 2^-110 a token, and room for
# the four products and sums of a step that each may round
def _small_v(tokens, largest=1.0):
    return tokens * 2.0 ** -108 * max(1.0, largest)


@pytest.mark.parametrize("dim,group,ratio", [(128, 32, 4), (64, 64, 16)])
@pytest.mark.parametrize("power", [-60, -80, -90, -98, -120])
def test_small_values_of_v(dim, group, ratio, power):
    """Few rows: at 2^-80 the roundings are all there is, further down there is an error that the
    header states."""
    rng = np.random.default_rng(-power)
    heads, page, nq, nkv = 2, 32, [1, 2, 1], [60, 700, 4000]
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group, vscale=2.0 ** power)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = _rand(rng, 4, heads * ratio, dim)
    out = _out(got, q, cu, nkv, table, max_q_len=2)
    o, most, mean = bounds.attention(want, 0, q, cu, nkv, table, 0, 0, dim ** -0.5)
    if power >= -80:
        bounds.check(out, o, most, mean)
    more = np.repeat([_small_v(m) for m in nkv], nq)[:, None, None]
    assert (np.abs(out - o) <= most + more).all()


def test_groups_of_v_of_different_size():
    """A group near 2^70 beside groups near 1: the small ones keep their bits."""
    rng = np.random.default_rng(1)
    heads, ratio, page, nkv, dim, group = 1, 4, 16, [50, 3000], 128, 32
    table, pages = _batch(rng, [1, 1], nkv, page)
    want, got = _pair(1, pages, page, heads, dim, group, fill=0xFF)
    for r, m in enumerate(nkv):
        x = np.arange(m)
        v = _rand(rng, m, heads, dim)
        v[:, :, 32:64] *= np.float32(2.0 ** 70)
        want.store(0, _rand(rng, m, heads, dim), ref.bf16_round(v), table[r][x // page] * page + x % page)
    _copy(want, got)
    q = _rand(rng, 2, ratio, dim)
    out = _out(got, q, [0, 1, 2], nkv, table, max_q_len=1)
    o, most, _ = bounds.attention(want, 0, q, [0, 1, 2], nkv, table, 0, 0, dim ** -0.5)
    more = np.array([_small_v(m, 2.0 ** 73) for m in nkv])[:, None, None]
    assert (np.abs(out - o) <= most + more).all()


@pytest.mark.parametrize("nq,nkv,ratio,page", [([1, 3], [500, 1333], 40, 16), ([1, 1], [700, 20], 300, 1024),
                                               ([2, 1, 5], [3, 2000, 40], 33, 1024), ([1, 2], [5000, 3000], 11, 1024),
                                               ([7], [2049], 129, 112)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5)])
def test_many_query_heads_and_large_pages(nq, nkv, ratio, page, window, sinks):
    """A token's query heads fill row tiles alone, or end inside one; pages larger than a tile."""
    rng = np.random.default_rng(ratio)
    heads, dim, group = 1, 64, 64
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = _rand(rng, int(cu[-1]), heads * ratio, dim)
    for most in (None, max(nq), 1000):
        out = _out(got, q, cu, nkv, table, window=window, sinks=sinks, max_q_len=most)
        bounds.check(out, *bounds.attention(want, 0, q, cu, nkv, table, window, sinks, dim ** -0.5))
