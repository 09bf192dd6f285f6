"""Eviction from the 4-bit paged cache on the GPU (weigh, choose_tokens, compact,
release_pages) against plain numpy (tests/evict_ref.py): weights within a bound that counts
roundings, everything else entry for entry and byte for byte."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import evict_ref as evict  # noqa: E402
import int4_ref as ref  # noqa: E402
from kv_cache_compression_03_gb300 import build, cachegen as cg  # noqa: E402

from test_gpu_int4 import FORMATS, _batch, _copy, _dev, _filled, _ints, _np, _pair, _rand, _same_bytes  # noqa: E402


def _floats(x):
    return torch.tensor(np.asarray(x, dtype=np.float32), device="cuda")


def _status(f, code):
    with pytest.raises(cg.CacheGenError) as e:
        f()
    assert e.value.status == code


# ------------------------------------------------------------------- weigh

# query tokens, cached tokens, query heads of a KV head: 1 to 8, 9 to 16 and more rows, one and
# several row tiles, requests without rows and without tokens, rows before the first token
WEIGHED = [([1] * 9, [1, 15, 16, 17, 128, 129, 700, 3100, 9001], 4),
           ([1, 1, 1], [33, 5000, 257], 1),
           ([4, 3, 0, 1], [4, 1500, 40, 9001], 3),
           ([16, 5, 0], [300, 16, 0], 4),
           ([70, 1, 33], [1025, 1, 400], 4),
           ([9, 300], [5, 513], 2)]


def _weigh_case(rng, nq, nkv, ratio, dim, group, page, heads=2, scale=1.0):
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group)
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int64)
    q = _rand(rng, int(cu[-1]), heads * ratio, dim, scale=scale)
    return table, want, got, cu, q


def _check_weights(out, before, want, tol):
    """out within tol of before + want where there is a token, untouched elsewhere."""
    there = ~np.isnan(want)
    over = np.abs(out[there] - before[there].astype(np.float64) - want[there]) - tol[there] - 2.0 ** -23 * np.abs(out[there])
    assert (over <= 0).all(), float(over.max())


@pytest.mark.parametrize("i", range(len(WEIGHED)))
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (129, 3), (700, 37)])
@pytest.mark.parametrize("dim,group,page", [(128, 32, 16), (64, 64, 48)])
def test_weigh(i, window, sinks, dim, group, page):
    nq, nkv, ratio = WEIGHED[i]
    rng = np.random.default_rng(7 * i + window)
    table, want, got, cu, q = _weigh_case(rng, nq, nkv, ratio, dim, group, page)
    width = table.shape[1] * page + 3
    before = np.abs(rng.standard_normal((len(nq), 2, width))).astype(np.float32)
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, window, sinks, dim ** -0.5, width)
    for most in (None, max(nq)):
        w = _floats(before)
        out = torch.full_like(w, -7.0)
        args = (_dev(q), _ints(cu), _ints(nkv), _ints(table))
        res = got.weigh(*args, w, window=window, sinks=sinks, max_q_len=most, out=out)
        assert res is out and torch.equal(w.cpu(), torch.from_numpy(before))
        got.check()
        _check_weights(out.cpu().numpy(), before, exact, tol)
        assert (out.cpu().numpy()[np.isnan(exact)] == -7.0).all()
        # in place, to the same bits
        assert got.weigh(*args, w, window=window, sinks=sinks, max_q_len=most) is w
        assert torch.equal(w[~torch.isnan(_floats(exact))], out[~torch.isnan(_floats(exact))])
        assert np.array_equal(w.cpu().numpy()[np.isnan(exact)], before[np.isnan(exact)])
        # from nothing: zeros, and each row's weights sum to one
        new = got.weigh(*args, window=window, sinks=sinks, max_q_len=most).cpu().numpy()
        assert new.shape == (len(nq), 2, table.shape[1] * page)
        for r, m in enumerate(nkv):
            sees = sum(min(m, max(0, m - nq[r] + 1 + k)) > 0 for k in range(nq[r]))
            assert np.allclose(new[r].sum(-1), ratio * sees, rtol=2.0 ** -12, atol=0)
            assert not new[r, :, m:].any()


@pytest.mark.parametrize("dim,group", [f for f in FORMATS if f not in ((128, 32), (64, 64))])
@pytest.mark.parametrize("i", [0, 2, 4])
def test_weigh_other_formats(dim, group, i):
    test_weigh(i, 0, 0, dim, group, 32)


@pytest.mark.parametrize("scale,qscale", [(0.0, 1.0), (-0.2, 1.0), (2.0 ** -130, 2.0 ** 100), (0.1, 2.0 ** -120)])
@pytest.mark.parametrize("nq", [1, 40])
def test_weigh_scales(scale, qscale, nq):
    rng = np.random.default_rng(5)
    table, want, got, cu, q = _weigh_case(rng, [nq], [400], 2, 64, 32, 16)
    q = ref.bf16_round(q * np.float32(qscale))
    exact, tol = evict.weigh(want, 0, q, cu, [400], table, 0, 0, scale, 400)
    out = got.weigh(_dev(q), _ints(cu), _ints([400]), _ints(table), scale=scale)
    got.check()
    _check_weights(out.cpu().numpy()[..., :400], np.zeros(exact.shape, np.float32), exact, tol)


@pytest.mark.parametrize("nq", [1, 70])
def test_weigh_of_channels_that_differ(nq):
    """Keys as models have them: a few channels many times as large as the others, which lo and s
    follow; the scores are sums of far smaller terms."""
    rng = np.random.default_rng(11)
    heads, dim, m, page = 2, 128, 2000, 16
    want, got = _pair(1, 125, page, heads, dim, 32)
    size = np.exp2(rng.integers(-2, 2, dim)) * np.where(np.arange(dim) % 32 == 3, 32, 1)
    k = ref.bf16_round((_rand(rng, m, heads, dim) * size).astype(np.float32))
    want.store(0, k, k, np.arange(m))
    _copy(want, got)
    q = ref.bf16_round((_rand(rng, nq, 4, dim) / size).astype(np.float32))
    table = np.arange(125)[None]
    exact, _ = evict.weigh(want, 0, q, [0, nq], [m], table, 0, 0, dim ** -0.5, m)
    out = got.weigh(_dev(q), _ints([0, nq]), _ints([m]), _ints(table)).cpu().numpy()
    # no sum here passes 2^7, so what cancels costs 2^-17 at most of the 30 roundings of 2^-24 each
    assert np.abs(out - exact).max() / exact.max() < 30 * 2.0 ** -17
    assert np.linalg.norm(out - exact) / np.linalg.norm(exact) < 2.0 ** -19


@pytest.mark.parametrize("low", [13, 14, 15, 79])
@pytest.mark.parametrize("more", [-1, 0, 1, 16])
@pytest.mark.parametrize("nq,ratio", [(4, 1), (2, 2), (8, 1), (20, 1)])
def test_weigh_where_the_windows_begin_at_the_last_of_the_first_tokens(low, more, nq, ratio):
    """The first row's window begins with token `low`, at a blob's end, the others' behind it; the tokens
    between, if they are not of the first ones, are seen by some rows only."""
    rng = np.random.default_rng(low)
    window, sinks = 400, low // 16 * 16 + 16 + more
    nkv = [window + nq - 1 + low]
    table, want, got, cu, q = _weigh_case(rng, [nq], nkv, ratio, 64, 32, 16)
    width = table.shape[1] * 16
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, window, sinks, 0.125, width)
    out = torch.zeros(1, 2, width, device="cuda")
    got.weigh(_dev(q), _ints(cu), _ints(nkv), _ints(table), out, window=window, sinks=sinks, max_q_len=nq)
    got.check()
    _check_weights(out.cpu().numpy(), np.zeros(out.shape, np.float32), exact, tol)


@pytest.mark.parametrize("nq,nkv,ratio,heads", [([200] * 4, [250, 200, 777, 201], 7, 8),    # 352 units of 128 rows
                                                 ([129], [3000], 1, 1),                     # 2 units, cut in pieces
                                                 ([65, 1, 0, 90], [65, 900, 30, 40], 3, 2),  # rows before the first token
                                                 ([33] * 3, [40, 1033, 129], 2, 3),          # 66 rows, few beside
                                                 ([700], [700], 5, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 17), (257, 3)])
@pytest.mark.parametrize("dim,group,page", [(128, 32, 64), (64, 32, 16), (128, 128, 48)])
def test_weigh_of_many_rows(nq, nkv, ratio, heads, window, sinks, dim, group, page):
    rng = np.random.default_rng(sum(nkv) + window + dim)
    table, want, got, cu, q = _weigh_case(rng, nq, nkv, ratio, dim, group, page, heads=heads)
    width = table.shape[1] * page
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, window, sinks, dim ** -0.5, width)
    out = torch.zeros(len(nq), heads, width, device="cuda")
    args = (_dev(q), _ints(cu), _ints(nkv), _ints(table))
    got.weigh(*args, out, window=window, sinks=sinks, max_q_len=max(nq))
    got.check()
    got_w = out.cpu().numpy()
    _check_weights(got_w, np.zeros_like(got_w), exact, tol)
    assert not got_w[np.isnan(exact)].any()
    # the weights of each row sum to one
    for r, m in enumerate(nkv):
        assert np.allclose(got_w[r].sum(-1), ratio * min(nq[r], m), rtol=2.0 ** -12, atol=0)
    norm = np.linalg.norm(np.nan_to_num(exact))
    assert np.linalg.norm(got_w - np.nan_to_num(exact)) / norm < 2.0 ** -19


def test_weigh_of_many_rows_reports_bad_pages():
    rng = np.random.default_rng(31)
    nq, m, page = 150, 900, 16
    table, want, got, cu, q = _weigh_case(rng, [nq], [m], 2, 64, 32, page)
    bad = table.copy()
    bad[0, [3, 20, 21]] = [1 << 20, -1, 1 << 30]
    out = got.weigh(_dev(q), _ints(cu), _ints([m]), _ints(bad)).cpu().numpy()
    _status(got.check, cg.CG_ERR_CORRUPT)
    gone = np.r_[48:64, 320:352]
    assert not out[0, :, gone].any() and np.isfinite(out).all()
    assert np.allclose(out[0].sum(-1), 2 * nq, rtol=2.0 ** -12)
    # as if those tokens were not there: the others' weights, renormalised row by row
    keep = np.delete(np.arange(m), gone)
    k, _, _ = want.values(0, table[0][keep // page] * page + keep % page)
    for h in range(2):
        exact = np.zeros(len(keep))
        for g in range(2):
            z = q[:, 2 * h + g].astype(np.float64) @ k[:, h].T * 0.125
            z = np.where(keep[None, :] <= (m - nq + np.arange(nq))[:, None], z, -np.inf)
            e = np.exp(z - z.max(1, keepdims=True))
            exact += (e / e.sum(1, keepdims=True)).sum(0)
        assert np.abs(out[0, h, keep] - exact).max() <= 2.0 ** -17 * exact.max()


def test_weigh_of_many_rows_reports_requests_that_share_rows():
    """Bounds of rows that go back and forth: every other request has all of them, more tiles of 128 than
    a batch of so many tokens."""
    rng = np.random.default_rng(41)
    nq, n = 600, 61
    table, want, got, cu, q = _weigh_case(rng, [nq], [nq], 2, 64, 32, 16)
    to_and_fro = [0, nq] * (n // 2) + [0, nq]
    w = torch.zeros(n, 2, table.shape[1] * 16, device="cuda")
    got.weigh(_dev(q), _ints(to_and_fro), _ints([nq] * n), _ints(np.repeat(table, n, 0)), w)
    _status(got.check, cg.CG_ERR_CORRUPT)
    a = got.weigh(_dev(q), _ints(cu), _ints([nq]), _ints(table))     # and the next call is right
    got.check()
    assert torch.allclose(a.sum(-1), torch.full((1, 2), 2.0 * nq, device="cuda"), rtol=2.0 ** -12)


@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("qscale", [1.0, 2.0 ** -100, 2.0 ** 60])
def test_weigh_of_many_rows_scales(scale, qscale):
    rng = np.random.default_rng(32)
    table, want, got, cu, q = _weigh_case(rng, [90], [300], 2, 64, 32, 16)
    q = ref.bf16_round(q * np.float32(qscale))
    exact, tol = evict.weigh(want, 0, q, cu, [300], table, 0, 0, scale / qscale, 300)
    out = got.weigh(_dev(q), _ints(cu), _ints([300]), _ints(table), scale=scale / qscale)
    got.check()
    _check_weights(out.cpu().numpy()[..., :300], np.zeros(exact.shape, np.float32), exact, tol)


def test_weigh_strides_layers_and_streams():
    rng = np.random.default_rng(9)
    nq, nkv, ratio, heads, dim, page = [1, 2], [300, 77], 4, 3, 64, 16
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, 32, layers=3, layer=2)
    cu = np.array([0, 1, 3])
    q = _rand(rng, 3, heads * ratio, dim)
    width = table.shape[1] * page
    exact, tol = evict.weigh(want, 2, q, cu, nkv, table, 0, 0, dim ** -0.5, width)
    wide_q = torch.zeros(3, heads * ratio + 2, dim + 8, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 1:-1, :dim] = _dev(q)
    wide_t = torch.full((2, table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide_t[:, :table.shape[1]] = _ints(table)
    base = torch.full((heads, 2, width + 9), 0.25, device="cuda")
    out = base.transpose(0, 1)[:, :, 2:2 + width]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in [None] + streams:
        base.fill_(0.25)
        torch.cuda.synchronize()
        got.weigh(wide_q[:, 1:-1, :dim], _ints(cu), _ints(nkv), wide_t[:, :table.shape[1]], out, layer=2, stream=s)
        torch.cuda.synchronize()
        got.check()
        o = out.cpu().numpy()
        _check_weights(o, np.full_like(o, 0.25), exact, tol)
        assert (o[np.isnan(exact)] == 0.25).all()
        assert (base[:, :, :2] == 0.25).all() and (base[:, :, 2 + width:] == 0.25).all()


@pytest.mark.parametrize("nq", [1, 30])
def test_weigh_reports_bad_requests_and_pages(nq):
    rng = np.random.default_rng(3)
    nkv, page = [100, 200, 130], 16
    table, want, got, cu, q = _weigh_case(rng, [nq] * 3, nkv, 2, 64, 32, page)
    width = table.shape[1] * page
    args = _dev(q), _ints(cu)
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, 0, 0, 0.125, width)

    def go(lens, tab=table, width=width, **kw):
        out = torch.full((3, 2, width), -7.0, device="cuda")
        got.weigh(*args, _ints(lens), _ints(tab), torch.zeros_like(out), out=out, **kw)
        return out.cpu().numpy()

    for lens, w in (([100, -1, 130], width), ([100, width + 1, 130], width), (nkv, 150)):
        out = go(lens, width=w)
        _status(got.check, cg.CG_ERR_CORRUPT)
        assert (out[1] == -7.0).all()
        for r in (0, 2):
            m = nkv[r]
            assert (np.abs(out[r, :, :m] - exact[r, :, :m]) <= tol[r, :, :m] + 2.0 ** -23).all()
    if nq > 1:
        out = go(nkv, max_q_len=nq - 1)
        _status(got.check, cg.CG_ERR_INVALID_ARG)
        assert (out == -7.0).all()
    # a page outside the cache: its tokens get nothing, the others all of it
    bad = table.copy()
    bad[1, 2] = 1 << 20
    out = go(nkv, bad)
    _status(got.check, cg.CG_ERR_CORRUPT)
    assert not out[1, :, 32:48].any()
    assert np.allclose(out[1, :, :200].sum(-1), 2 * nq, rtol=2.0 ** -12)


@pytest.mark.parametrize("nq", [1, 40, 150])
def test_weigh_of_bounds_of_rows_that_do_not_ascend(nq):
    """The requests that they leave, whose rows follow one another, are right; the others' weights stay as they were."""
    rng = np.random.default_rng(nq)
    nkv = [nq + 300, nq + 7, nq + 500, nq]
    table, want, got, cu, q = _weigh_case(rng, [nq] * 4, nkv, 2, 64, 32, 16)
    width = table.shape[1] * 16
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, 0, 0, 0.125, width)
    for at, right in (([0, 1, 2, 3, 5], [0, 1, 2]), ([0, 1, 2, 3, 2], [0, 1, 2]), ([0, 1, 2, 3, -1], [0, 1, 2]),
                      ([0, 9, 2, 3, 4], [2, 3]), ([0, 1, -3, 3, 4], [0, 3]), ([0, 1, 2, 1 << 22, 4], [0, 1])):
        out = torch.full((4, 2, width), -7.0, device="cuda")
        got.weigh(_dev(q), _ints(np.array(at) * nq), _ints(nkv), _ints(table), out=out)
        _status(got.check, cg.CG_ERR_CORRUPT)
        o = out.cpu().numpy()
        for r in range(4):
            if r in right:
                m = nkv[r]
                assert (np.abs(o[r, :, :m] - exact[r, :, :m]) <= tol[r, :, :m] + 2.0 ** -23 * o[r, :, :m]).all(), (at, r)
                assert (o[r, :, m:] == -7.0).all()
            else:
                assert (o[r] == -7.0).all(), (at, r)


def test_weigh_without_rows_or_requests():
    rng = np.random.default_rng(3)
    table, want, got, cu, q = _weigh_case(rng, [0, 0], [40, 0], 2, 64, 32, 16)
    w = _floats(rng.random((2, 2, 48)))
    out = torch.full_like(w, -7.0)
    empty = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    got.weigh(empty, _ints([0, 0, 0]), _ints([40, 0]), _ints(table), w, out=out)
    got.check()
    assert torch.equal(out[0, :, :40], w[0, :, :40]) and (out[0, :, 40:] == -7.0).all() and (out[1] == -7.0).all()
    none = got.weigh(empty, _ints([0]), _ints([]), _ints(np.empty((0, 3))))
    assert none.shape == (0, 2, 48)
    # rows without room for a token: a request that has one is reported, whatever else there is
    no_room = torch.empty(2, 2, 0, device="cuda")
    got.weigh(_dev(q[:0]), _ints([0, 0, 0]), _ints([0, 0]), _ints(table), no_room)
    got.check()
    got.weigh(_dev(q[:0]), _ints([0, 0, 0]), _ints([40, 0]), _ints(table), no_room)
    _status(got.check, cg.CG_ERR_CORRUPT)
    # padding: rows of q behind the last request's, pages that are not there
    q = _dev(_rand(rng, 5, 4, 64))
    a = got.weigh(q[:2], _ints([0, 2, 2]), _ints([40, 0]), _ints(table))
    b = got.weigh(q, _ints([0, 2, 2]), _ints([40, 0]), _ints(table), max_q_len=2)
    got.check()
    assert torch.equal(a, b)


def test_weigh_from_nothing_into_rows_without_room():
    rng = np.random.default_rng(3)
    _, _, got, _, _ = _weigh_case(rng, [0, 0], [40, 0], 2, 64, 32, 16)
    q, lens = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), _ints([0, 0])
    none = got.weigh(q, _ints([0, 0, 0]), lens, _ints(np.empty((2, 0))))          # a table of no pages
    assert none.shape == (2, 2, 0)
    out = torch.empty(2, 2, 0, device="cuda")
    assert got.weigh(q, _ints([0, 0, 0]), lens, _ints([[1], [0]]), out=out) is out
    got.check()


def test_weigh_with_tables_and_rows_of_other_widths():
    """The same call but for how far its table and its weights reach."""
    rng = np.random.default_rng(21)
    nkv = [40, 33]
    table, want, got, cu, q = _weigh_case(rng, [1, 1], nkv, 4, 64, 32, 16)
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, 0, 0, 0.125, 64)
    for wide, width in ((3, 40), (3, 64), (200, 40), (4000, 64), (4000, 60000), (3, 40)):
        t = np.full((2, wide), -1, np.int32)
        t[:, :3] = table[:, :3]
        w = torch.zeros(2, 2, width, device="cuda")
        got.weigh(_dev(q), _ints(cu), _ints(nkv), _ints(t), w, max_q_len=1)
        got.check()
        out = w.cpu().numpy()
        for r, m in enumerate(nkv):
            assert (np.abs(out[r, :, :m] - exact[r, :, :m]) <= tol[r, :, :m] + 2.0 ** -23).all()
            assert not out[r, :, m:].any()


@pytest.mark.parametrize("nq,ratio", [(1, 4), (2, 4), (9, 1), (30, 2), (300, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5)])
def test_weigh_with_and_without_room_for_scores(nq, ratio, window, sinks):
    """Rows of weights so wide that scores cannot be stored for the batch: computed twice instead, with the same result."""
    rng = np.random.default_rng(nq)
    nkv = [nq + 700, nq, nq + 33]
    table, want, got, cu, q = _weigh_case(rng, [nq] * 3, nkv, ratio, 128, 64, 16)
    wide = np.full((3, 1 << 19), -1, np.int32)     # 2^23 tokens a row: 800 MB of scores for 6 lists and 4 rows,
    wide[:, :table.shape[1]] = table               # 1.2 GB of sums for 36 tiles of 128 rows
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, window, sinks, 128 ** -0.5, table.shape[1] * 16)
    kw = dict(window=window, sinks=sinks, max_q_len=nq)
    few = got.weigh(_dev(q), _ints(cu), _ints(nkv), _ints(table), **kw).cpu().numpy()
    base = torch.zeros(3, 2, 1 << 23, device="cuda")
    got.weigh(_dev(q), _ints(cu), _ints(nkv), _ints(wide), base, **kw)
    got.check()
    many = base[..., :few.shape[-1]].cpu().numpy()
    assert not base[..., few.shape[-1]:].any()
    for out in (few, many):
        _check_weights(out, np.zeros_like(out), exact, tol)


@pytest.mark.parametrize("n", [33, 300])
def test_weigh_many_requests(n):
    rng = np.random.default_rng(n)
    nkv = [1 + (37 * i) % 90 for i in range(n)]
    nq = [min(k, i % 3) for i, k in enumerate(nkv)]
    table, want, got, cu, q = _weigh_case(rng, nq, nkv, 2, 64, 64, 16)
    width = table.shape[1] * 16
    exact, tol = evict.weigh(want, 0, q, cu, nkv, table, 0, 0, 0.125, width)
    out = got.weigh(_dev(q), _ints(cu), _ints(nkv), _ints(table), max_q_len=2).cpu().numpy()
    got.check()
    _check_weights(out, np.zeros_like(out), exact, tol)


@pytest.mark.parametrize("nq,ratio", [(1, 4), (40, 4)])
def test_weigh_gives_the_same_bits_in_graphs_and_on_streams(nq, ratio):
    rng = np.random.default_rng(2)
    nkv = [9001, 4000, 17 + nq]
    table, want, got, cu, q = _weigh_case(rng, [nq] * 3, nkv, ratio, 128, 32, 16)
    args = (_dev(q), _ints(cu), _ints(nkv), _ints(table))
    first = got.weigh(*args, max_q_len=nq)
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, outs = [], []
    for s in streams[:2]:
        g, out = torch.cuda.CUDAGraph(), torch.zeros_like(first)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            got.weigh(*args, max_q_len=nq, out=out)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = got.weigh(*args, max_q_len=nq, stream=streams[2])
        torch.cuda.synchronize()
        for o in outs + [eager]:
            assert torch.equal(o, first)
    got.check()


def test_weigh_of_more_units_than_blocks_gives_the_same_bits():
    """672 units of 128 rows, of odd and even numbers of tiles: whichever blocks take them, and in whatever order."""
    rng = np.random.default_rng(17)
    nq, nkv, heads, ratio = [700, 333, 512, 90, 1000], [1100, 333, 900, 700, 1000], 8, 4
    table, want, got, cu, q = _weigh_case(rng, nq, nkv, ratio, 64, 32, 16, heads=heads)
    assert sum(-(-n * ratio // 128) for n in nq) * heads > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    args = (_dev(q), _ints(cu), _ints(nkv), _ints(table))
    first = got.weigh(*args, max_q_len=max(nq))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(40):   # one at a time, and beside one another
        outs = [got.weigh(*args, max_q_len=max(nq), stream=s) for s in streams[:1 + i % 3]]
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, first)
    got.check()


@pytest.mark.parametrize("nq,ratio", [(1, 4), (40, 4)])
def test_a_wait_of_weigh_that_runs_out_is_reported(nq, ratio):
    variant = build.build_test_variant("test_cg_test_attn_timeout", ["CG_TEST_ATTN_TIMEOUT"])
    rng = np.random.default_rng(nq)
    table, want, got, cu, q = _weigh_case(rng, [nq] * 2, [9001, 8000], ratio, 64, 32, 64)
    args = (_dev(q), _ints(cu), _ints([9001, 8000]), _ints(table))
    before = got.weigh(*args, max_q_len=nq)
    got.check()
    with cg.use_library(variant):
        got.weigh(*args, max_q_len=nq)
        _status(got.check, cg.CG_ERR_TIMEOUT)
    assert torch.equal(got.weigh(*args, max_q_len=nq), before)
    got.check()


# ------------------------------------------------------------------ choose

@pytest.mark.parametrize("layers,lens,width,budget,recent,sinks", [
    (None, [0, 1, 5, 40], 40, 5, 2, 1), (None, [3000, 100, 2999], 3100, 100, 0, 0), (2, [5000, 4096], 5000, 1024, 1020, 4),
    (3, [65, 64, 63, 1], 65, 64, 8, 3), (1, [70000], 70001, 3000, 64, 16), (2, [500, 7], 600, 0, 0, 0),
    (2, [20000], 20000, 19999, 5, 5), (None, [33], 33, 200, 100, 7), (4, [9000] * 3, 9000, 1, 0, 0),
    # by a warp, four and eight of them; by a block's digits from 152 rows on; by a cluster; from memory
    (7, [128, 127, 1], 128, 31, 1, 2), (3, [512, 290, 511], 512, 100, 0, 37), (2, [2048, 1500, 513], 2048, 700, 64, 0),
    (None, [5120, 2049], 5120, 2000, 3, 3), (None, [8192, 5121], 8192, 100, 0, 1), (38, [2500, 2049], 2600, 1000, 7, 4),
    (39, [8192, 6000], 8192, 64, 0, 0), (None, [98304], 98304, 500, 20, 2), (None, [140000, 9], 150000, 1024, 100, 4)])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
def test_choose(layers, lens, width, budget, recent, sinks, kind):
    rng = np.random.default_rng(sum(lens) + budget)
    shape = ((layers,) if layers else ()) + (len(lens), 2, width)
    w = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 3, shape).astype(np.float32)
    elif kind == "odd":
        w = np.where(rng.random(shape) < 0.3, rng.choice([0.0, -0.0, np.nan, np.inf, -np.inf, -1.0, 1e-45, -1e-45], shape), w)
        w = w.astype(np.float32)
    kept, new = evict.choose(w, lens, budget, recent, sinks)
    got = cg.choose_tokens(_floats(w), _ints(lens), budget, recent=recent, sinks=sinks)
    got.check()
    assert np.array_equal(got.lens.cpu().numpy(), new)
    assert np.array_equal(got.kept.cpu().numpy(), kept)


# the widest rows that a cluster holds (131072: 8 blocks of 512 threads, 32 tokens each), and the next
@pytest.mark.parametrize("lens,width,budget,recent,sinks", [
    ([98305, 90001], 98305, 4096, 64, 4), ([131072, 131071], 131072, 4000, 256, 16), ([131072], 131072, 130000, 0, 0),
    ([131073, 131072], 131073, 4096, 64, 4)])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
def test_choose_from_the_widest_rows(lens, width, budget, recent, sinks, kind):
    test_choose(None, lens, width, budget, recent, sinks, kind)


def test_choose_strides_out_graph_and_bad_lengths():
    rng = np.random.default_rng(1)
    base = _floats(rng.random((3, 4, 2, 210)))
    w = base.transpose(0, 1)[:, 1:, :, 5:205]         # [4 layers, 2 requests, 2 heads, 200]
    lens = _ints([150, 60])
    kept, new = evict.choose(w.cpu().numpy(), [150, 60], 70, 10, 4)
    out = cg.choose_tokens(w, lens, 70, 10, 4, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    out.check()
    assert np.array_equal(out.kept.cpu().numpy(), kept)
    # lengths in place, in a graph
    plan = cg.KeptTokens(torch.empty_like(out.kept), lens, out.status)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cg.choose_tokens(w, lens, 70, 10, 4, out=plan)
    g.replay()
    plan.check()
    assert lens.tolist() == [70, 60] and np.array_equal(plan.kept.cpu().numpy(), kept)
    got = cg.choose_tokens(w, _ints([201, 60]), 70, 10, 4)
    _status(got.check, cg.CG_ERR_CORRUPT)
    assert got.lens.tolist() == [201, 60] and (got.kept[:, 0] == -1).all()
    assert np.array_equal(got.kept[:, 1].cpu().numpy(), kept[:, 1])
    got = cg.choose_tokens(w, _ints([150, -3]), 70, 10, 4)
    _status(got.check, cg.CG_ERR_CORRUPT)
    assert got.lens.tolist() == [70, -3] and np.array_equal(got.kept[:, 0].cpu().numpy(), kept[:, 0])
    none = cg.choose_tokens(w[:, :0], _ints([]), 3)
    none.check()
    assert none.kept.shape == (4, 0, 2, 3)


# ----------------------------------------------------------------- compact

def _random_kept(rng, layers, lens, heads, budget):
    kept = np.full((layers, len(lens), heads, budget), -1, np.int32)
    new = np.array([min(m, budget) for m in lens], np.int32)
    for l, r, h in np.ndindex(*kept.shape[:3]):
        kept[l, r, h, :new[r]] = np.sort(rng.permutation(lens[r])[:new[r]])
    return kept, new


def _random_cache(rng, layers, lens, heads, dim, group, page):
    """Any bytes will do: the move does not look at them."""
    held = [-(-m // page) for m in lens]
    pages = sum(held) + 2
    want, got = _pair(layers, pages, page, heads, dim, group)
    want.data[:] = rng.integers(0, 256, want.data.shape, dtype=np.uint8)
    _copy(want, got)
    ids = rng.permutation(pages)
    table = np.full((len(lens), max(held + [1]) + 1), -1, np.int32)
    for r, n in enumerate(held):
        table[r, :n] = ids[sum(held[:r]):sum(held[:r]) + n]
    return want, got, table


@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("lens,budget,page", [([1, 2, 33, 17], 16, 16), ([500, 3, 130], 97, 48), ([1100], 1023, 64),
                                              ([700, 700], 350, 1024), ([64, 65, 48], 48, 16)])
def test_compact(dim, group, lens, budget, page):
    rng = np.random.default_rng(dim + group + budget)
    heads, layers = 3, 2
    want, got, table = _random_cache(rng, layers + 1, lens, heads, dim, group, page)
    kept, new = _random_kept(rng, layers, lens, heads, budget)
    width = max(lens) + 5
    w = rng.random((layers, len(lens), heads, width)).astype(np.float32)
    wt = _floats(w)
    got.compact(_ints(kept), _ints(new), _ints(lens), _ints(table), weights=wt, layer=1)
    got.check()
    evict.compact(want, 1, kept, new, lens, table, w)
    _same_bytes(want, got)
    assert np.array_equal(wt.cpu().numpy(), w)


def test_compact_leaves_what_stays_in_place():
    """A front that two requests share, all of whose tokens stay, and requests that lose nothing or all."""
    rng = np.random.default_rng(4)
    heads, dim, group, page = 2, 64, 32, 16
    lens, new = [100, 90, 40, 50], np.array([60, 50, 40, 0], np.int32)
    want, got, table = _random_cache(rng, 1, lens, heads, dim, group, page)
    table[1, :2] = table[0, :2]      # 32 shared tokens
    kept = np.full((1, 4, heads, 70), -1, np.int32)
    for r, h in np.ndindex(2, heads):
        n, m = int(new[r]), lens[r]
        kept[0, r, h, :n] = np.concatenate([np.arange(32 + h), np.sort(32 + h + rng.permutation(m - 32 - h)[:n - 32 - h])])
    kept[0, 2] = 1 << 30             # not looked at
    got.compact(_ints(kept[0]), _ints(new), _ints(lens), _ints(table))
    got.check()
    kept[0, 2, :, :40] = np.arange(40)
    evict.compact(want, 0, kept, new, lens, table)
    _same_bytes(want, got)


def test_compact_strides_streams_and_graph():
    rng = np.random.default_rng(6)
    lens, budget, page = [300, 200], 128, 32
    want, got, table = _random_cache(rng, 2, lens, 2, 128, 64, page)
    kept, new = _random_kept(rng, 2, lens, 2, budget)
    wide = torch.full((2, 2, 2, budget + 6), 77, dtype=torch.int32, device="cuda").transpose(0, 2)
    wide[..., 3:3 + budget] = _ints(kept)
    base = _floats(rng.random((2, 2, 2, 330)))
    w = base.transpose(0, 1)
    w0 = w.cpu().numpy().copy()
    args = (wide[..., 3:3 + budget], _ints(new), _ints(lens), _ints(table))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got.compact(*args, weights=w)
    for call in (g.replay, lambda: got.compact(*args, weights=w, stream=torch.cuda.Stream())):
        call()
        torch.cuda.synchronize()
        got.check()
        evict.compact(want, 0, kept, new, lens, table, w0)
        _same_bytes(want, got)
        assert np.array_equal(w.cpu().numpy(), w0)


@pytest.mark.parametrize("what", ["falls", "equal", "negative", "beyond", "minus one", "too many", "longer", "table", "weights",
                                  "new negative"])
def test_compact_refuses_what_it_is_not_given_right(what):
    rng = np.random.default_rng(8)
    lens, budget, page, heads = [100, 90], 40, 16, 2
    want, got, table = _random_cache(rng, 1, lens, heads, 64, 64, page)
    kept, new = _random_kept(rng, 1, lens, heads, budget)
    w = rng.random((1, 2, heads, 100)).astype(np.float32)
    lens_in, new_in, wt = list(lens), list(new), _floats(w)
    whole = what in ("too many", "longer", "table", "weights", "new negative")
    if what == "falls":
        kept[0, 0, 1, 7], kept[0, 0, 1, 8] = kept[0, 0, 1, 8], kept[0, 0, 1, 7]
    elif what == "equal":
        kept[0, 0, 1, 8] = kept[0, 0, 1, 7]
    elif what == "negative":
        kept[0, 0, 1, 0] = -2
    elif what == "beyond":
        kept[0, 0, 1, 39] = 100
    elif what == "minus one":
        kept[0, 0, 1, 39] = -1
    elif what == "too many":
        new_in[0] = 41
    elif what == "longer":
        new_in[0] = 101
    elif what == "table":
        lens_in[0] = table.shape[1] * page + 1
    elif what == "weights":
        wt = wt[..., :95].contiguous()
    else:
        new_in[0] = -1
    got.compact(_ints(kept), _ints(new_in), _ints(lens_in), _ints(table), weights=wt)
    _status(got.check, cg.CG_ERR_CORRUPT)
    got.check()
    # the head (or request) at fault stays, all others move
    good = kept.copy()
    good[0, 0] = _random_kept(rng, 1, lens, heads, budget)[0][0, 0]
    before = want.data.copy()
    evict.compact(want, 0, good, new, lens, table, w)
    bad_heads = range(heads) if whole else [1]
    for h in range(heads):
        if h in bad_heads:
            want.data[0, table[0, :7], h] = before[0, table[0, :7], h]
        else:
            pages = table[0, :7]
            redo = ref.Cache(*want.shape)
            redo.data[:] = before
            evict.compact(redo, 0, kept, new, lens, table)
            want.data[0, pages, h] = redo.data[0, pages, h]
    _same_bytes(want, got)


def test_compact_reports_pages_outside_the_cache():
    rng = np.random.default_rng(8)
    lens, budget, page = [100], 50, 16
    want, got, table = _random_cache(rng, 1, lens, 1, 64, 32, page)
    kept, new = _random_kept(rng, 1, lens, 1, budget)
    bad = table.copy()
    bad[0, 4] = 1 << 25           # tokens 64 .. 79 cannot be read: their places keep what they had
    got.compact(_ints(kept), _ints(new), _ints(lens), _ints(bad))
    _status(got.check, cg.CG_ERR_CORRUPT)
    start = ref.Cache(*want.shape)
    start.data[:] = want.data
    evict.compact(want, 0, kept, new, lens, table)
    for i, j in enumerate(kept[0, 0, 0]):
        if 64 <= j < 80:
            blob, at = evict._token(want, 0, 0, int(table[0, i // page]) * page + i % page)
            old, _ = evict._token(start, 0, 0, int(table[0, i // page]) * page + i % page)
            blob[at] = old[at]
    _same_bytes(want, got)


def _move(cache, first_layer, kept, new_lens, lens, table, weights):
    """evict.compact, all tokens of a list at once."""
    D, g, page = cache.dim, cache.dim // cache.group, cache.page
    a = 8 * D + 64 * g

    def places(r, j):   # page, blob, bytes of the tokens
        slot = table[r][j // page].astype(np.int64) * page + j % page
        tok = slot[:, None] % 16
        v = a + tok // 2 * D + 2 * (tok % 2) + np.arange(D).reshape(-1, 4)[:, :2].reshape(-1)
        at = np.concatenate([tok * (D // 2) + np.arange(D // 2), 8 * D + tok * 4 * g + np.arange(4 * g), v,
                             a + 8 * D + tok * 4 * g + np.arange(4 * g)], 1)
        return slot[:, None] // page, slot[:, None] % page // 16, at

    for l, r, h in np.ndindex(*kept.shape[:3]):
        n, m = int(new_lens[r]), int(lens[r])
        if n == m:
            continue
        data, src = cache.data[first_layer + l], kept[l, r, h, :n].astype(np.int64)
        p, b, at = places(r, src)
        got = data[p, h, b, at].copy()
        p, b, at = places(r, np.arange(n))
        data[p, h, b, at] = got
        w = weights[l, r, h, src].copy()
        weights[l, r, h, :m] = 0
        weights[l, r, h, :n] = w


def test_numpy_moves_agree():
    rng = np.random.default_rng(1)
    want, got, table = _random_cache(rng, 1, [70, 40], 2, 64, 32, 16)
    kept, new = _random_kept(rng, 1, [70, 40], 2, 33)
    a, b = rng.random((1, 2, 2, 70)), None
    b, other = a.copy(), ref.Cache(*want.shape)
    other.data[:] = want.data
    evict.compact(want, 0, kept, new, [70, 40], table, a)
    _move(other, 0, kept, new, [70, 40], table, b)
    assert np.array_equal(want.data, other.data) and np.array_equal(a, b)


# layers, requests, heads, tokens, those that stay: a block to a list, and clusters of two, four and eight to one, each in
# more rounds of 128 tokens to a block than it reads ahead; lists of odd lengths
@pytest.mark.parametrize("layers,requests,heads,top,budget,blocks", [
    (5, 8, 4, 1500, 1301, 1), (1, 10, 12, 3100, 2700, 4), (2, 2, 1, 9000, 7999, 8), (1, 1, 1, 9000, 8000, 8),
    (1, 152, 1, 700, 655, 1), (1, 151, 1, 2800, 2577, 4), (1, 100, 1, 2300, 2100, 4), (1, 99, 1, 4500, 4201, 8)])
@pytest.mark.parametrize("how", ["random", "one goes early", "one goes late", "from within a blob"])
def test_compact_in_rounds(layers, requests, heads, top, budget, blocks, how):
    rng = np.random.default_rng(top + budget)
    dim, group, page = 64, 32, 48
    lists, size = layers * requests * heads, 1
    while size < 8 and lists < 152 and lists * size < 400:
        size *= 2
    assert size == blocks and budget > 4 * 128 * blocks   # the case is what it says: five rounds at least
    lens = [top - (i * 37) % max(1, (top - budget) // 2) for i in range(requests)]
    want, got, table = _random_cache(rng, layers, lens, heads, dim, group, page)
    if how in ("random", "from within a blob"):
        kept, new = _random_kept(rng, layers, lens, heads, budget)
        if how == "from within a blob":   # the first stay in place, 13 of a blob's tokens among them
            first = 16 * 40 + 13
            for l, r, h in np.ndindex(*kept.shape[:3]):
                kept[l, r, h, :first] = np.arange(first)
                kept[l, r, h, first:] = first + 1 + np.sort(rng.permutation(lens[r] - first - 1)[:budget - first])
    else:
        at = 5 if how == "one goes early" else budget - 70
        kept = np.broadcast_to(np.delete(np.arange(budget + 1, dtype=np.int32), at), (layers, requests, heads, budget)).copy()
        new = np.full(requests, budget, np.int32)
    w = rng.random((layers, requests, heads, top + 3)).astype(np.float32)
    wt = _floats(w)
    got.compact(_ints(kept), _ints(new), _ints(lens), _ints(table), weights=wt)
    got.check()
    _move(want, 0, kept, new, lens, table, w)
    _same_bytes(want, got)
    assert np.array_equal(wt.cpu().numpy(), w)


def test_pages_of_a_layer_behind_4_gib():
    """Offsets into a layer that pass 32 bits, second layer of two: weights, attention with shared tokens and the move."""
    rng = np.random.default_rng(15)
    heads, dim, group, page, shared, lens, budget = 8, 128, 32, 64, 128, [700, 260], 400
    table, pages = _batch(rng, [1, 1], lens, page)
    table[1, :shared // page] = table[0, :shared // page]
    want, _ = _filled(rng, lens, table, pages, page, heads, dim, group)
    bytes_of_page = want.data[0, 0].size
    far = (1 << 32) // bytes_of_page + 3                     # pages of a layer before the first of these
    got = cg.Int4Cache(2, far + pages, page, heads, dim, group,
                       data=torch.empty(2 * (far + pages) * bytes_of_page, dtype=torch.uint8, device="cuda"))
    there = got.data.view(2, far + pages, -1)[1, far:]
    there.copy_(torch.from_numpy(want.data[0].reshape(pages, -1)))
    at = np.where(table >= 0, table + far, -1)
    q, cu, kw = _rand(rng, 2, 4 * heads, dim), np.arange(3), dict(layer=1, max_q_len=1)
    args = (_dev(q), _ints(cu), _ints(lens), _ints(at))
    w = got.weigh(*args, **kw)
    exact, tol = evict.weigh(want, 0, q, cu, lens, table, 0, 0, dim ** -0.5, w.shape[2])
    _check_weights(w.cpu().numpy(), np.zeros(w.shape, np.float32), exact, tol)
    out = got.attention(*args, shared=shared, **kw)
    o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, dim ** -0.5)
    assert (np.abs(_np(out) - o) <= tol).all()
    many = _rand(rng, 260, 4 * heads, dim)                   # and of many rows
    out = got.attention(_dev(many), _ints([0, 130, 260]), _ints(lens), _ints(at), shared=shared, layer=1)
    o, tol = ref.attention(want, 0, many, [0, 130, 260], lens, table, 0, 0, dim ** -0.5)
    assert (np.abs(_np(out) - o) <= tol).all()
    w = got.weigh(_dev(many), _ints([0, 130, 260]), _ints(lens), _ints(at), layer=1)
    exact, tol = evict.weigh(want, 0, many, [0, 130, 260], lens, table, 0, 0, dim ** -0.5, w.shape[2])
    _check_weights(w.cpu().numpy(), np.zeros(w.shape, np.float32), exact, tol)
    kept, new = _random_kept(rng, 1, lens, heads, budget)
    kept[..., :shared] = np.arange(shared)                   # the shared pages stay as they are
    for h in range(heads):
        kept[0, 0, h, shared:] = shared + np.sort(rng.permutation(lens[0] - shared)[:budget - shared])
    kept[0, 1, :, :lens[1]] = np.arange(lens[1])
    got.compact(_ints(kept[0]), _ints(new), _ints(lens), _ints(at), layer=1)
    got.check()
    _move(want, 0, kept, new, lens, table, np.zeros((1, 2, heads, 700)))
    assert np.array_equal(there.cpu().numpy(), want.data[0].reshape(pages, -1))


def test_compact_and_choose_of_nothing():
    rng = np.random.default_rng(8)
    want, got, table = _random_cache(rng, 1, [20], 2, 64, 32, 16)
    got.compact(torch.empty((1, 2, 0), dtype=torch.int32, device="cuda"), _ints([0]), _ints([20]), _ints(table))
    got.compact(torch.empty((0, 2, 4), dtype=torch.int32, device="cuda"), _ints([]), _ints([]), _ints(table[:0]))
    got.compact(torch.empty((0, 1, 2, 4), dtype=torch.int32, device="cuda"), _ints([0]), _ints([20]), _ints(table))
    got.check()
    _same_bytes(want, got)


# ----------------------------------------------------------------- release

@pytest.mark.parametrize("n,top,page", [(1, 40, 16), (5, 100, 16), (64, 4000, 16), (300, 500, 64), (2000, 90, 48), (8192, 40, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_pages(n, top, page, in_place):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, top + 1, n)
    new = np.minimum(lens, rng.integers(0, top + 1, n))
    held = -(-lens // page)
    table = np.full((n, max(int(held.max()), 1) + 2), -5, np.int32)
    ids = rng.permutation(int(held.sum()) + 9)
    at = 0
    for r, k in enumerate(held):
        table[r, :k] = ids[at:at + k]
        at += k
    free = np.full(int(held.sum()) + 9 + 3, -7, np.int32)
    free[:9] = ids[at:]
    want_t, want_f, want_n, cu = evict.release(table, lens, new, free, 9, page)
    t, f, count, l, nl = _ints(table), _ints(free), _ints([9]), _ints(lens), _ints(new)
    out = None
    if in_place:
        out = cg.ReleasePlan(torch.empty(n + 1, dtype=torch.int32, device="cuda"), l if n % 2 else nl, count,
                             torch.empty(16, dtype=torch.uint8, device="cuda"))
    p = cg.release_pages(t, l, nl, f, count, page, num_pages=int(held.sum()) + 9, out=out)
    p.check()
    assert np.array_equal(t.cpu().numpy(), want_t) and np.array_equal(f.cpu().numpy(), want_f)
    assert p.free_count.item() == want_n and np.array_equal(p.cu.cpu().numpy(), cu)
    assert np.array_equal(p.lens.cpu().numpy(), new)


@pytest.mark.parametrize("what,code", [("negative", cg.CG_ERR_INVALID_ARG), ("longer", cg.CG_ERR_INVALID_ARG),
                                       ("list", cg.CG_ERR_CAPACITY), ("table", cg.CG_ERR_CAPACITY),
                                       ("count", cg.CG_ERR_CORRUPT), ("count below", cg.CG_ERR_CORRUPT)])
def test_release_pages_takes_all_or_nothing(what, code):
    table = np.arange(20, dtype=np.int32).reshape(4, 5)
    lens, new, free, count = [80, 70, 5, 0], [16, 0, 5, 0], np.full(30, -7), 3
    if what == "negative":
        new[2] = -1
    elif what == "longer":
        new[3] = 1
    elif what == "list":
        free = free[:11]
    elif what == "table":
        lens[1] = 81
    elif what == "count":
        count = 31
    else:
        count = -1
    t, f = _ints(table), _ints(free)
    p = cg.release_pages(t, _ints(lens), _ints(new), f, _ints([count]), 16)
    _status(p.check, code)
    assert np.array_equal(t.cpu().numpy(), table) and (f == -7).all()
    assert p.free_count.item() == count and not p.cu.any() and p.lens.tolist() == lens


def test_release_pages_reports_page_ids_outside_the_cache():
    table = _ints([[4, 99, 2], [-1, 3, 0]])
    f = _ints([-7] * 8)
    p = cg.release_pages(table, _ints([48, 20]), _ints([16, 0]), f, _ints([0]), 16, num_pages=10)
    _status(p.check, cg.CG_ERR_CORRUPT)
    assert f.tolist() == [99, 2, -1, 3] + [-7] * 4 and p.free_count.item() == 4
    assert table.tolist() == [[4, -1, -1], [-1, -1, 0]]
    none = cg.release_pages(table[:0], _ints([]), _ints([]), f, _ints([2]), 16)
    none.check()
    assert none.free_count.item() == 2 and none.cu.tolist() == [0]


# ------------------------------------------------------------ all together

def test_requests_that_share_a_front_are_cut_and_attended():
    """Three requests on 64 shared tokens, cut to a budget that keeps those, and attended with shared=:
    the shared pages are read by all and written by none."""
    rng = np.random.default_rng(13)
    heads, ratio, dim, group, page, shared = 2, 4, 64, 64, 16, 64
    own = [200, 90, 130]
    lens = [shared + n for n in own]
    held = [-(-n // page) for n in own]
    pages = 4 + sum(held) + 1
    want, got = _pair(1, pages, page, heads, dim, group)
    ids = rng.permutation(pages)
    table = np.full((3, 4 + max(held)), -1, np.int32)
    table[:, :4], at = ids[:4], 4
    for r, n in enumerate(held):
        table[r, 4:4 + n] = ids[at:at + n]
        at += n
        x = np.arange(lens[r])[0 if r == 0 else shared:]
        want.store(0, _rand(rng, len(x), heads, dim), _rand(rng, len(x), heads, dim), table[r][x // page] * page + x % page)
    _copy(want, got)
    q, cu = _rand(rng, 3, heads * ratio, dim), np.arange(4)
    tab, dq, dcu = _ints(table), _dev(q), _ints(cu)
    w = got.weigh(dq, dcu, _ints(lens), tab, max_q_len=1)
    exact, tol = evict.weigh(want, 0, q, cu, lens, table, 0, 0, dim ** -0.5, w.shape[2])
    _check_weights(w.cpu().numpy(), np.zeros(w.shape, np.float32), exact, tol)
    before = w.cpu().numpy()[None].copy()
    c = cg.choose_tokens(w, _ints(lens), 150, recent=20, sinks=shared)
    kept, new = evict.choose(before, lens, 150, 20, shared)
    assert np.array_equal(c.kept.cpu().numpy(), kept[0]) and np.array_equal(c.lens.cpu().numpy(), new)
    got.compact(c.kept, c.lens, _ints(lens), tab, weights=w)
    got.check()
    front = want.data[0, table[0, :4]].copy()
    evict.compact(want, 0, kept, new, lens, table, before)
    assert np.array_equal(want.data[0, table[0, :4]], front)
    _same_bytes(want, got)
    out = got.attention(dq, dcu, c.lens, tab, max_q_len=1, shared=shared)
    got.check()
    o, tol = ref.attention(want, 0, q, cu, new, table, 0, 0, dim ** -0.5)
    assert (np.abs(_np(out) - o) <= tol).all()
    free, count = _ints([-7] * pages), _ints([0])
    rel = cg.release_pages(tab, _ints(lens), c.lens, free, count, page, num_pages=pages)
    rel.check()
    # at its end a request gives back its own pages, the last one all of them
    for r in range(3):
        ends = [0 if i == r == 2 else shared if i <= r else n for i, n in enumerate(new)]
        was = rel.lens.clone()
        rel = cg.release_pages(tab, was, _ints(ends), free, rel.free_count, page, num_pages=pages)
        rel.check()
    assert sorted(free[:int(rel.free_count)].tolist()) == sorted(ids[:at].tolist())


def test_a_cache_is_kept_to_its_budget():
    """grow -> store -> attention and weigh, step by step in a graph; then choose -> compact -> release in
    another; then on with what stayed, as if the other tokens had never been there."""
    rng = np.random.default_rng(12)
    layers, heads, ratio, dim, group, page, budget = 2, 2, 4, 64, 32, 16, 40
    n, width, pages = 3, 8, 30
    cache = cg.Int4Cache(layers, pages, page, heads, dim, group)
    want = ref.Cache(layers, pages, page, heads, dim, group)
    table, lens = _ints(np.full((n, width), -1)), _ints([0] * n)
    free, count = _ints(np.arange(pages)), _ints([pages])
    counts = _ints([1, 1, 1])
    weights = torch.zeros(layers, n, heads, width * page, device="cuda")
    sums = np.zeros(weights.shape)
    k = torch.empty(layers, 2 * n, heads, dim, dtype=torch.bfloat16, device="cuda")
    v, q = torch.empty_like(k), torch.empty(2 * n, heads * ratio, dim, dtype=torch.bfloat16, device="cuda")
    e = torch.empty
    plan = cg.PagePlan(_ints([0] * (2 * n)), _ints([0] * (n + 1)), lens, count, e(16, dtype=torch.uint8, device="cuda"))
    out = torch.zeros(layers, 2 * n, heads * ratio, dim, dtype=torch.bfloat16, device="cuda")

    def step():
        cg.grow_pages(table, lens, counts, free, count, page, 2 * n, num_pages=pages, out=plan)
        cache.store(k, v, plan.slots)
        for l in range(layers):
            cache.attention(q, plan.cu, lens, table, layer=l, out=out[l], max_q_len=2)
            cache.weigh(q, plan.cu, lens, table, weights[l], layer=l, max_q_len=2)

    def cut():
        c = cg.choose_tokens(weights, lens, budget, recent=8, sinks=2)
        cache.compact(c.kept, c.lens, lens, table, weights=weights)
        rel = cg.ReleasePlan(e(n + 1, dtype=torch.int32, device="cuda"), lens, count, e(16, dtype=torch.uint8, device="cuda"))
        cg.release_pages(table, lens, c.lens, free, count, page, num_pages=pages, out=rel)
        return c, rel

    s = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0], stream=s):
        step()
    with torch.cuda.graph(graphs[1], stream=s):
        c, rel = cut()
    held = [0] * n
    for i in range(70):
        news = [1 + (i + r) % 2 for r in range(n)]
        total = sum(news)
        hk, hv = _rand(rng, layers, 2 * n, heads, dim), _rand(rng, layers, 2 * n, heads, dim)
        hq = _rand(rng, 2 * n, heads * ratio, dim)
        k.copy_(_dev(hk)), v.copy_(_dev(hv)), q.copy_(_dev(hq)), counts.copy_(_ints(news))
        graphs[0].replay()
        plan.check(), cache.check()
        held = [a + b for a, b in zip(held, news)]
        assert lens.tolist() == held
        slots, tab = plan.slots.cpu().numpy(), table.cpu().numpy()
        cu = np.concatenate([[0], np.cumsum(news)])
        for l in range(layers):
            want.store(l, hk[l], hv[l], slots)
            o, tol = ref.attention(want, l, hq[:total], cu, held, tab, 0, 0, dim ** -0.5)
            assert (np.abs(_np(out[l])[:total] - o) <= tol).all()
            w, tol = evict.weigh(want, l, hq[:total], cu, held, tab, 0, 0, dim ** -0.5, width * page)
            got = weights[l].cpu().numpy()
            there = ~np.isnan(w)
            sums[l][there] += w[there]
            # the bound of this step on top of what the earlier ones were off (counted anew each step)
            assert (np.abs(got[there] - sums[l][there]) <= tol[there] + 2.0 ** -22 * got[there]).all()
            assert not got[~there].any()
            sums[l] = got
        if i % 20 == 19:
            before = weights.cpu().numpy().copy()
            kept, new = evict.choose(before, held, budget, 8, 2)
            nfree = int(count.item())
            _, want_f, want_n, _ = evict.release(tab, held, new, free.cpu().numpy(), nfree, page)
            graphs[1].replay()
            c.check(), cache.check(), rel.check()
            assert np.array_equal(c.kept.cpu().numpy(), kept) and lens.tolist() == new.tolist()
            evict.compact(want, 0, kept, new, held, tab, before)
            _same_bytes(want, cache)
            assert np.array_equal(weights.cpu().numpy(), before)
            assert np.array_equal(free.cpu().numpy(), want_f) and int(count.item()) == want_n
            held, sums = new.tolist(), before.astype(np.float64)
