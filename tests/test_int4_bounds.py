"""The bounds of tests/int4_bounds.py: results rounded to bf16 keep them, and an oracle that
loses one blob, one tile or one token does not."""
import numpy as np
import pytest

import int4_bounds as bounds
import int4_ref as ref


def _filled(rng, nkv, dim, group, heads, page=16, whole=False):
    held = [-(-m // page) for m in nkv]
    ids = rng.permutation(sum(held) + 2)
    table = np.full((len(nkv), max(held)), -1, np.int32)
    cache = ref.Cache(1, sum(held) + 2, page, heads, dim, group)
    at = 0
    for r, m in enumerate(nkv):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
        x = np.arange(m)
        k = rng.standard_normal((m, heads, dim)) * np.exp(0.7 * rng.standard_normal((heads, dim)))
        v = bounds.whole_numbers(rng, m, heads, dim, group=group) if whole else rng.standard_normal((m, heads, dim)) + 0.5
        cache.store(0, ref.bf16_round(k.astype(np.float32)), ref.bf16_round(v.astype(np.float32)),
                    table[r][x // page] * page + x % page)
    return cache, table


def _refused(f):
    with pytest.raises(AssertionError):
        f()


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32)])
@pytest.mark.parametrize("nq,n", [(4, 700), (13, 3100), (64, 2055)])
def test_random_data(dim, group, nq, n):
    rng = np.random.default_rng(nq + dim)
    nkv, cu = [n, n - 11], [0, nq, 2 * nq]
    cache, table = _filled(rng, nkv, dim, group, 1)
    q = ref.bf16_round(rng.standard_normal((2 * nq, 8, dim)).astype(np.float32))
    args = cache, 0, q, cu, nkv, table, 0, 0, dim ** -0.5
    o, most, mean = bounds.attention(*args)
    want, wide = ref.attention(*args)
    assert np.allclose(o, want, rtol=1e-9, atol=1e-12) and ((most <= wide) | ~np.isfinite(most)).all()
    bounds.check(ref.bf16_round(o.astype(np.float32)), o, most, mean)
    for lose in (np.arange(32, 48), np.arange(n - 32, n - 16), np.arange(128, 256)):
        less = bounds.attention(*args, lose=lose)[0]
        _refused(lambda: bounds.check(ref.bf16_round(less.astype(np.float32)), o, most, mean))


@pytest.mark.parametrize("n,window,sinks", [(40, 0, 0), (700, 0, 0), (3100, 0, 0), (3100, 700, 9)])
def test_whole_numbers(n, window, sinks):
    rng = np.random.default_rng(n)
    cache, table = _filled(rng, [n], 64, 32, 2, whole=True)
    args = cache, 0, [0, 3], [n], table, window, sinks, 2, 2
    o, tol = bounds.counted(*args)
    plain = ref.attention(cache, 0, np.zeros((3, 4, 64), np.float32), [0, 3], [n], table, window, sinks, 0.1)[0]
    assert np.allclose(o, plain, atol=1e-12)
    assert (np.abs(ref.bf16_round(o.astype(np.float32)) - o) <= tol).all()
    low = max(0, n - 3 + 1 - window) if window else 0
    for lost in (low + 2, low + 16, n - 20, n - 4) + ((0, sinks - 1) if sinks else ()):
        less = ref.bf16_round(bounds.counted(*args, lose=[lost])[0].astype(np.float32))
        assert (np.abs(less - o) > tol).any((1, 2)).all()   # a single token, in every row
