"""Attention over the 4-bit cache with tokens that all requests share (attention(shared=)),
against the formula in 64 bits (tests/int4_ref.py) and the call without."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_ref as ref  # noqa: E402
from kv_cache_compression_03_gb300 import build, cachegen as cg  # noqa: E402

from test_gpu_int4 import FORMATS, _copy, _dev, _ints, _np, _pair, _rand  # noqa: E402


@pytest.fixture(autouse=True, params=["by size", "two passes"])
def passes(request):
    """As the sizes have it (the shared tokens here are few), and the shared tokens always in a pass of their own."""
    if request.param == "by size":
        yield
    else:
        with cg.use_library(build.build_test_variant("test_cg_test_shared_two", ["CG_TEST_SHARED_TWO"])):
            yield


def _case(rng, nq, own, shared, heads, ratio, dim, group, page, layers=1, layer=0, scale=1.0, fill=0xFF):
    """Requests with `own` tokens behind `shared` common ones; unused places hold bytes that are no numbers."""
    held = [-(-k // page) for k in own]
    front = shared // page
    pages = front + sum(held) + 1
    want, got = _pair(layers, pages, page, heads, dim, group, fill)
    ids = rng.permutation(pages)
    table = np.full((len(own), front + max(held)), -1, np.int32)
    table[:, :front] = ids[:front]
    at = front
    for r, n in enumerate(held):
        table[r, front:front + n] = ids[at:at + n]
        at += n
    for r, n in enumerate(own):
        x = np.arange(shared + n)[0 if r == 0 else shared:]
        if len(x):
            want.store(layer, _rand(rng, len(x), heads, dim, scale=scale), _rand(rng, len(x), heads, dim),
                       table[r][x // page] * page + x % page)
    _copy(want, got)
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int64)
    q = _rand(rng, int(cu[-1]), heads * ratio, dim)
    return table, want, got, cu, q, [shared + n for n in own]


# new tokens, own tokens, shared ones, query heads of a KV head: few and many rows on either side
SHAPES = [([1] * 5, [1, 17, 40, 300, 2], 96, 1), ([1] * 3, [5, 1, 700], 4800, 4), ([1] * 12, list(range(1, 13)), 960, 4),
          ([4, 2, 0, 3], [4, 900, 0, 3], 1920, 4), ([20, 1, 7], [20, 1, 300], 480, 4), ([150, 40], [150, 200], 960, 2),
          ([1] * 70, [1 + i for i in range(70)], 192, 2), ([1], [1], 96, 8), ([300], [300], 4800, 2)]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("dim,group,page", [(128, 32, 16), (64, 64, 48)])
def test_shared_tokens(i, dim, group, page):
    nq, own, shared, ratio = SHAPES[i]
    rng = np.random.default_rng(i + dim)
    table, want, got, cu, q, lens = _case(rng, nq, own, shared, 2, ratio, dim, group, page)
    o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, dim ** -0.5)
    for most in (None, max(nq)):
        out = got.attention(_dev(q), _ints(cu), _ints(lens), _ints(table), max_q_len=most, shared=shared)
        got.check()
        over = np.abs(_np(out) - o) - tol
        assert (over <= 0).all(), float(over.max())
    # entries of the other rows are not read, nor is what lies behind a row's last page
    other = table.copy()
    other[1:, :shared // page] = 1 << 29
    again = got.attention(_dev(q), _ints(cu), _ints(lens), _ints(other), max_q_len=max(nq), shared=shared)
    got.check()
    assert torch.equal(again, out)


@pytest.mark.parametrize("dim,group", [f for f in FORMATS if f not in ((128, 32), (64, 64))])
@pytest.mark.parametrize("i", [1, 4])
def test_shared_tokens_other_formats(dim, group, i):
    test_shared_tokens(i, dim, group, 32)


@pytest.mark.parametrize("scale,qscale", [(0.0, 1.0), (-0.2, 1.0), (2.0 ** -26, 2.0 ** 23)])
@pytest.mark.parametrize("i", [0, 5, 6, 8])
def test_scales(scale, qscale, i):
    """Scales that the kernel for many rows takes into Q: the two passes' maxima are still of one kind."""
    nq, own, shared, ratio = SHAPES[i]
    rng = np.random.default_rng(i)
    table, want, got, cu, q, lens = _case(rng, nq, own, shared, 2, ratio, 64, 32, 16)
    q = ref.bf16_round(q * np.float32(qscale))
    o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, scale)
    out = got.attention(_dev(q), _ints(cu), _ints(lens), _ints(table), scale=scale, max_q_len=max(nq), shared=shared)
    got.check()
    assert (np.abs(_np(out) - o) <= tol).all()


@pytest.mark.parametrize("nq,n", [(1, 3), (1, 40), (70, 2)])
def test_weights_on_either_side(nq, n):
    """Scores that put nearly all weight on the shared tokens, or nearly none."""
    rng = np.random.default_rng(nq + n)
    heads, dim, page, shared = 1, 64, 16, 64
    for side in (0, 1):
        table, want, got, cu, q, lens = _case(rng, [nq] * n, [nq + 9] * n, shared, heads, 2, dim, 32, page)
        q = np.abs(q)
        big = np.full((1, heads, dim), 6.0, np.float32)
        slots = [table[0, 0] * page + 3] if side == 0 else [table[r, shared // page] * page for r in range(n)]
        for s in slots:   # position 3, or each request's first own token: seen by every query
            want.store(0, big, _rand(rng, 1, heads, dim), [s])
        _copy(want, got)
        o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, 1.0)
        out = got.attention(_dev(q), _ints(cu), _ints(lens), _ints(table), scale=1.0, shared=shared)
        got.check()
        assert (np.abs(_np(out) - o) <= tol).all()


def test_layers_strides_streams_and_rows_behind_the_last():
    rng = np.random.default_rng(3)
    nq, own, shared, heads, ratio, dim, page = [1, 2], [30, 9], 64, 3, 2, 64, 16
    table, want, got, cu, q, lens = _case(rng, nq, own, shared, heads, ratio, dim, 32, page, layers=3, layer=1)
    o, tol = ref.attention(want, 1, q, cu, lens, table, 0, 0, dim ** -0.5)
    wide = torch.zeros(5, heads * ratio + 1, dim + 8, dtype=torch.bfloat16, device="cuda")
    wide[:3, 1:, 8:] = _dev(q)
    base = torch.full((heads * ratio, 5, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    out = base.transpose(0, 1)
    for s in (None, torch.cuda.Stream()):
        base.fill_(3.0)
        torch.cuda.synchronize()
        got.attention(wide[:, 1:, 8:], _ints(cu), _ints(lens), _ints(table), layer=1, out=out, stream=s, shared=shared)
        torch.cuda.synchronize()
        got.check()
        assert (np.abs(_np(out)[:3] - o) <= tol).all() and (out[3:] == 3.0).all()


@pytest.mark.parametrize("nq", [1, 40])
def test_errors(nq):
    rng = np.random.default_rng(3)
    table, want, got, cu, q, lens = _case(rng, [nq] * 3, [nq + 5] * 3, 64, 2, 2, 64, 32, 16)
    width = table.shape[1] * 16
    o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, 0.125)

    def go(lens, tab=table, **kw):
        out = torch.full((3 * nq, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        got.attention(_dev(q), _ints(cu), _ints(lens), _ints(tab), out=out, shared=64, **kw)
        return _np(out)

    # not long enough for its new tokens, longer than its row, negative: that request alone is left out
    for bad, code in ((64 + nq - 1, cg.CG_ERR_INVALID_ARG), (10, cg.CG_ERR_INVALID_ARG), (width + 1, cg.CG_ERR_CORRUPT),
                      (-1, cg.CG_ERR_CORRUPT)):
        out = go([lens[0], bad, lens[2]])
        with pytest.raises(cg.CacheGenError) as e:
            got.check()
        assert e.value.status == code
        assert (out[nq:2 * nq] == 3.0).all()
        keep = np.r_[0:nq, 2 * nq:3 * nq]
        assert (np.abs(out[keep] - o[keep]) <= tol[keep]).all()
    # a shared page outside the cache: nobody sees its tokens
    bad = table.copy()
    bad[:, 1] = 1 << 24
    out = go(lens, bad)
    with pytest.raises(cg.CacheGenError) as e:
        got.check()
    assert e.value.status == cg.CG_ERR_CORRUPT
    cut = np.delete(table, 1, 1)   # the same tokens without that page
    o2, tol2 = ref.attention(want, 0, q, cu, [m - 16 for m in lens], cut, 0, 0, 0.125)
    assert (np.abs(out - o2) <= tol2).all()
    for kw in (dict(shared=8), dict(shared=-16), dict(shared=width + 16), dict(shared=64, window=100), dict(shared=1 << 32)):
        with pytest.raises(ValueError):
            got.attention(_dev(q), _ints(cu), _ints(lens), _ints(table), **kw)


@pytest.mark.parametrize("nq", [1, 40])
def test_bounds_of_rows_that_do_not_ascend(nq, monkeypatch):
    """Whichever requests they leave without fault are right, the rows of the others stay as they were, also where
    the workspace held something else before."""
    rng = np.random.default_rng(nq)
    table, want, got, cu, q, lens = _case(rng, [nq] * 4, [nq + 5, nq, nq + 30, nq + 1], 960, 2, 2, 64, 32, 16)
    o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, 0.125)
    empty = torch.empty

    def of_no_numbers(*a, **k):
        t = empty(*a, **k)
        return t.fill_(0xFF) if t.dtype is torch.uint8 else t

    monkeypatch.setattr(torch, "empty", of_no_numbers)
    # the bounds, in rows of a request, and the requests that they leave
    for at, right in (([0, 1, 2, 3, 5], [0, 1, 2]), ([0, 1, 2, 3, 2], [0, 1]), ([0, 1, 2, 3, -1], []),
                      ([0, 9, 2, 3, 4], [2, 3]), ([0, 1, -3, 3, 4], [0, 3]), ([0, 1, 2, 1 << 25, 4], [0, 1]),
                      ([0, 1, 2, 3, 0], [])):
        out = torch.full((4 * nq, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        got.attention(_dev(q), _ints(np.array(at) * nq), _ints(lens), _ints(table), out=out, shared=960)
        with pytest.raises(cg.CacheGenError) as e:
            got.check()
        assert e.value.status == cg.CG_ERR_CORRUPT
        out = _np(out)
        for r in range(4):
            rows = slice(r * nq, (r + 1) * nq)
            if r in right:
                assert (np.abs(out[rows] - o[rows]) <= tol[rows]).all(), (at, r)
            else:
                assert (out[rows] == 3.0).all(), (at, r)


def _pieces(units, tiles, items, blocks):
    """Into how many pieces each unit of shared tokens is cut: the longest block's time counts, a piece's being its
    tiles and three more."""
    can = [s for s in range(1, 32) if s == 1 or (s <= tiles // 2 and units * s <= items)]
    return min(can, key=lambda s: (-(-units * s // blocks) * (-(-tiles // s) + 3), s))


# new tokens of each request, KV heads, shared tokens: 100 units of 256 rows each, cut in three. Two full row
# tiles to a unit; one row tile, whose softmax groups take turns at five tiles; the two kinds by turns
@pytest.mark.parametrize("nq,heads,shared", [([640, 640], 20, 1536), ([50, 50], 100, 1920), ([100, 200], 50, 1920)])
def test_more_pieces_than_blocks(nq, heads, shared):
    rng = np.random.default_rng(heads)
    blocks = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    units = -(-sum(nq) // 256) * heads
    pieces = _pieces(units, shared // 128, min(max(units * 31, 160), 640), blocks)
    assert pieces == 3 and units * pieces > blocks
    table, want, got, cu, q, lens = _case(rng, nq, [n + 9 for n in nq], shared, heads, 1, 64, 32, 64)
    o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, 0.125)
    args = (_dev(q), _ints(cu), _ints(lens), _ints(table))
    out = got.attention(*args, shared=shared, max_q_len=max(nq))
    got.check()
    over = np.abs(_np(out) - o) - tol
    assert (over <= 0).all(), float(over.max())
    for _ in range(5):
        assert torch.equal(got.attention(*args, shared=shared, max_q_len=max(nq)), out)
    got.check()


@pytest.mark.parametrize("nq,n", [(1, 3), (1, 40), (70, 2)])
@pytest.mark.parametrize("vscale", [2.0 ** 92, 2.0 ** -100])
def test_values_to_the_ends_of_the_range(nq, n, vscale):
    """V below 2^96 (2^92 times what no normal draw of these few passes), and small ones."""
    rng = np.random.default_rng(nq + n)
    heads, dim, page, shared = 2, 64, 16, 960
    table, want, got, cu, q, lens = _case(rng, [nq] * n, [nq + 9] * n, shared, heads, 2, dim, 32, page)
    for r, m in enumerate(lens):
        x = np.arange(m)[0 if r == 0 else shared:]
        v = _rand(rng, len(x), heads, dim, scale=vscale)
        assert np.abs(v).max() < 16 * vscale
        want.store(0, _rand(rng, len(x), heads, dim), v, table[r][x // page] * page + x % page)
    _copy(want, got)
    o, tol = ref.attention(want, 0, q, cu, lens, table, 0, 0, 0.125)
    out = got.attention(_dev(q), _ints(cu), _ints(lens), _ints(table), max_q_len=nq, shared=shared)
    got.check()
    # small values: the codes of the kernel for few rows are summed in units that end at 2^-106
    assert (np.abs(_np(out) - o) <= tol + 2.0 ** -108 * max(lens)).all()


@pytest.mark.parametrize("nq,n", [(1, 5), (1, 30), (50, 3)])
def test_the_same_bits_in_graphs_and_on_streams(nq, n):
    rng = np.random.default_rng(2)
    table, want, got, cu, q, lens = _case(rng, [nq] * n, [nq + 40 * i for i in range(n)], 3200, 2, 4, 128, 32, 16)
    args = (_dev(q), _ints(cu), _ints(lens), _ints(table))
    kw = dict(max_q_len=nq, shared=3200)
    first = got.attention(*args, **kw)
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for s in streams[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(got.attention(*args, **kw))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = got.attention(*args, **kw, stream=streams[2])
        torch.cuda.synchronize()
        for o in outs + [eager]:
            assert torch.equal(o, first)
    got.check()


def test_a_wait_that_runs_out_is_reported():
    variant = build.build_test_variant("test_cg_test_attn_timeout", ["CG_TEST_ATTN_TIMEOUT"])
    rng = np.random.default_rng(2)
    table, want, got, cu, q, lens = _case(rng, [1] * 20, [40] * 20, 9600, 2, 4, 64, 32, 64)
    args = (_dev(q), _ints(cu), _ints(lens), _ints(table))
    before = got.attention(*args, max_q_len=1, shared=9600)
    got.check()
    got._sizes.clear()                 # this variant takes two passes, and room for them
    with cg.use_library(variant):
        got.attention(*args, max_q_len=1, shared=9600)
        with pytest.raises(cg.CacheGenError) as e:
            got.check()
        assert e.value.status == cg.CG_ERR_TIMEOUT
    assert torch.equal(got.attention(*args, max_q_len=1, shared=9600), before)
    got.check()
