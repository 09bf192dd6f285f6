"""The 4-bit paged cache on the GPU: stored bytes and loaded values bit for
bit, page tables and slot maps entry for entry, attention within a bound that
counts its roundings, all against plain numpy (tests/int4_ref.py)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_ref as ref  # noqa: E402
from kv_cache_compression_03_gb300 import cachegen as cg  # noqa: E402
from kv_cache_compression_03_gb300 import synthetic  # noqa: E402

FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def _dev(x):
    """fp32 array of bf16 values -> bf16 tensor."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def _np(t):
    return t.float().cpu().numpy()


def _ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), dtype=torch.int32, device="cuda")


def _rand(rng, *shape, scale=1.0):
    return ref.bf16_round((rng.standard_normal(shape) * scale).astype(np.float32))


def _pair(layers, pages, page, heads, dim, group, fill=0):
    """The same cache in numpy and on the GPU (the latter's bytes are copied over by _copy)."""
    want = ref.Cache(layers, pages, page, heads, dim, group, fill)
    got = cg.Int4Cache(layers, pages, page, heads, dim, group,
                       data=torch.full((want.data.size,), fill, dtype=torch.uint8, device="cuda"))
    return want, got


def _copy(want, got):
    got.data.copy_(torch.from_numpy(want.data.reshape(-1)))


def _same_bytes(want, got):
    assert np.array_equal(got.data.cpu().numpy(), want.data.reshape(-1))


# ------------------------------------------------------------- store, load

@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("layers,tokens,heads,page", [(1, 1, 1, 16), (2, 37, 3, 48), (3, 130, 8, 64)])
def test_store_and_load(dim, group, layers, tokens, heads, page):
    rng = np.random.default_rng(dim + group + tokens)
    pages = tokens // page + 2
    want, got = _pair(layers + 1, pages, page, heads, dim, group, fill=0xA5)
    k = _rand(rng, layers, tokens, heads, dim) * np.exp2(rng.integers(-3, 4, (heads, dim)))
    v = _rand(rng, layers, tokens, heads, dim)
    k, v = ref.bf16_round(k), ref.bf16_round(v)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    slots[tokens // 2::7] = -1
    got.store(_dev(k), _dev(v), _ints(slots), layer=1)
    for i in range(layers):
        want.store(1 + i, k[i], v[i], slots)
    _same_bytes(want, got)   # other slots, padding and layer 0 untouched
    lk, lv = got.load(_ints(slots), layer=1, layers=layers)
    for i in range(layers):
        hold = slots >= 0
        wk, wv, _ = want.values(1 + i, slots[hold])
        for w, l in ((wk, lk[i]), (wv, lv[i])):
            l = _np(l)
            # s n is exact in fp32 and lo + s n then rounds as in fp32
            assert np.array_equal(ref.bits(l[hold]), ref.bits(ref.bf16_round(w.astype(np.float32))))
            assert not l[~hold].any()
    got.check()


def test_store_rows_that_need_care():
    """Constant rows, zeros of both signs, ties, subnormals, a range that only just fits, far offsets."""
    dim, group = 64, 32
    rows = np.zeros((10, 1, dim), np.float32)
    rows[1] = 7.25
    rows[2, :, ::2] = -0.0
    rows[3] = np.arange(dim) % 16              # s = 1: exact codes
    rows[4] = (np.arange(dim) % 31) * 0.5      # s = 1: halves, ties to even
    rows[5] = 100 + (np.arange(dim) % 4) * 0.5
    rows[6] = np.where(np.arange(dim) % 2, 1.0, -1.0) * 1.69e38
    rows[7] = (np.arange(dim) % 9) * 2.0 ** -133
    rows[8] = np.where(np.arange(dim) == 3, 3.0e38, 1e-30)
    rows[9] = -1e-38 * (np.arange(dim) % 3)
    rows = ref.bf16_round(rows)
    want, got = _pair(1, 1, 16, 1, dim, group)
    slots = np.arange(10)
    got.store(_dev(rows), _dev(rows[::-1].copy()), _ints(slots))
    want.store(0, rows, rows[::-1], slots)
    _same_bytes(want, got)
    got.check()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan, "overflow"])
def test_store_reports_what_it_cannot_hold(bad):
    rng = np.random.default_rng(3)
    k = _rand(rng, 4, 2, 64)
    v = _rand(rng, 4, 2, 64)
    if bad == "overflow":
        k[2, 1, 40], k[2, 1, 41] = ref.bf16_round(np.float32([3.3e38, -3.3e38]))
    else:
        k[2, 1, 40] = bad
    want, got = _pair(1, 1, 16, 2, 64, 32)
    got.store(_dev(k), _dev(v), _ints(np.arange(4)))
    want.store(0, k, v, np.arange(4))   # that group as zeros, all others as ever
    _same_bytes(want, got)
    with pytest.raises(cg.CacheGenError) as e:
        got.check()
    assert e.value.status == cg.CG_ERR_NONFINITE
    got.check()                         # raised once, then cleared


def test_store_reports_values_that_round_to_infinity():
    """lo + 15 s past bf16's largest value: the group is refused, so that no stored value is infinite."""
    rows = np.zeros((3, 1, 64), np.float32)
    # a range of 254.25 or 254.75 2^120 has s = 17 2^120: 255.75 2^120 rounds to 2^128, 255.25 2^120 does not
    rows[0, :, :32], rows[1, :, :32] = 0.75 * 2.0 ** 120, 0.25 * 2.0 ** 120
    rows[:2, :, 9] = 255 * 2.0 ** 120
    rows[2, :, 5] = 3.0e38
    rows = ref.bf16_round(rows)
    n, s, lo = ref.quantise(rows, 32)
    assert s[0, 0, 0] == 0 and s[1, 0, 0] == 17 * 2.0 ** 120 and s[2, 0, 0] > 0
    want, got = _pair(1, 1, 16, 1, 64, 32)
    got.store(_dev(rows), _dev(rows), _ints([0, 1, 2]))
    want.store(0, rows, rows, [0, 1, 2])
    _same_bytes(want, got)
    assert torch.isfinite(got.load(_ints([0, 1, 2]))[0].float()).all()
    with pytest.raises(cg.CacheGenError) as e:
        got.check()
    assert e.value.status == cg.CG_ERR_NONFINITE


def test_store_and_load_report_slots_outside_the_cache():
    rng = np.random.default_rng(4)
    k, v = _rand(rng, 3, 1, 64), _rand(rng, 3, 1, 64)
    want, got = _pair(1, 2, 16, 1, 64, 64)
    for wrong in (32, -2, 2 ** 31 - 1, -2 ** 31):
        slots = np.array([5, wrong, 31], np.int32)
        got.store(_dev(k), _dev(v), _ints(slots))
        want.store(0, k[[0, 2]], v[[0, 2]], slots[[0, 2]])
        _same_bytes(want, got)
        with pytest.raises(cg.CacheGenError) as e:
            got.check()
        assert e.value.status == cg.CG_ERR_CORRUPT
        a, b = got.load(_ints(slots))
        assert not _np(a)[1].any() and not _np(b)[1].any() and _np(a)[2].any()
        with pytest.raises(cg.CacheGenError):
            got.check()


def test_store_and_load_strided_rows():
    """K and V as parts of a wider projection, load into halves of a codec blob."""
    rng = np.random.default_rng(5)
    T, H, D = 21, 2, 128
    wide = _rand(rng, T, 3 * H + 4, D)
    w = _dev(wide)
    want, got = _pair(2, 2, 16, H, D, 64)
    slots = np.arange(T) + 3
    got.store(w[:, 4:4 + H], w[:, 5 + H:5 + 2 * H], _ints(slots), layer=1)
    want.store(1, wide[:, 4:4 + H], wide[:, 5 + H:5 + 2 * H], slots)
    _same_bytes(want, got)
    kv = torch.zeros(2, 2, T, H, D, dtype=torch.bfloat16, device="cuda")
    got.load(_ints(slots), layers=2, k_out=kv[:, 0], v_out=kv[:, 1])
    a, b = got.load(_ints(slots), layer=1)
    assert torch.equal(kv[1, 0], a) and torch.equal(kv[1, 1], b) and not kv[0].any()
    # heads before tokens
    t = _dev(wide).transpose(0, 1).contiguous().transpose(0, 1)
    got.data.zero_()
    got.store(t[:, 4:4 + H], t[:, 5 + H:5 + 2 * H], _ints(slots), layer=1)
    _same_bytes(want, got)
    got.store(w[:0, :H], w[:0, :H], _ints([]))
    assert got.load(_ints([]))[0].shape == (0, H, D)
    _same_bytes(want, got)


# ------------------------------------------------------------------- pages

def _grow_ref(table, lens, counts, free, nfree, page, tokens):
    table, slots, k = table.copy(), [], 0
    for r, (n, c) in enumerate(zip(lens, counts)):
        held = -(-n // page)
        for i in range(held, -(-(n + c) // page)):
            table[r, i] = free[nfree - 1 - k]
            k += 1
        slots += [table[r, x // page] * page + x % page for x in range(n, n + c)]
    return table, slots + [-1] * (tokens - len(slots)), nfree - k


@pytest.mark.parametrize("n,top,most,page", [(1, 0, 1, 16), (1, 40, 0, 16), (3, 100, 40, 48),
                                             (64, 500, 1, 16), (1025, 90, 3, 16),
                                             (300, 1000, 100, 64), (8192, 50, 9, 32), (2, 5, 9000, 16)])
def test_grow_pages(n, top, most, page):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, top + 1, n)
    counts = rng.integers(0, most + 1, n) if n > 2 else np.full(n, most)
    width = -(-int((lens + counts).max()) // page) + 1
    held, need = -(-lens // page), -(-(lens + counts) // page)
    total = int(need.sum())
    ids = rng.permutation(total + 5).astype(np.int32)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for r in range(n):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    free = np.concatenate([ids[at:], np.full(3, -7, np.int32)])   # 3 places behind the count
    nfree, tokens = len(free) - 3, int(counts.sum()) + 5
    t = _ints(table)
    p = cg.grow_pages(t, _ints(lens), _ints(counts), _ints(free), _ints([nfree]), page, tokens,
                      num_pages=total + 5)
    p.check()
    wt, ws, wf = _grow_ref(table, lens.tolist(), counts.tolist(), free, nfree, page, tokens)
    assert np.array_equal(t.cpu().numpy(), wt)
    assert p.slots.tolist() == ws
    assert p.cu.tolist() == [0] + np.cumsum(counts).tolist()
    assert p.lens.tolist() == (lens + counts).tolist()
    assert p.free_count.tolist() == [wf]


@pytest.mark.parametrize("what,code", [("pages", cg.CG_ERR_CAPACITY), ("width", cg.CG_ERR_CAPACITY),
                                       ("slots", cg.CG_ERR_CAPACITY), ("len", cg.CG_ERR_INVALID_ARG),
                                       ("count", cg.CG_ERR_INVALID_ARG), ("list", cg.CG_ERR_CORRUPT)])
@pytest.mark.parametrize("tokens", [60, 9000])
def test_grow_pages_takes_all_or_nothing(what, code, tokens):
    lens, counts, nfree, width = [5, 20, 0], [3, 30, 7], 6, 4
    if what == "pages":
        nfree = 2        # three are needed
    elif what == "width":
        width = 3
    elif what == "slots":
        counts[1], width, nfree = tokens, 9999, 6
    elif what == "len":
        lens[2] = -1
    elif what == "count":
        counts[0] = -3
    elif what == "list":
        nfree = 9
    table = np.full((3, width), 2, np.int32)
    t, l, c = _ints(table), _ints(lens), _ints(counts)
    p = cg.grow_pages(t, l, c, _ints(range(8)), _ints([nfree]), 16, tokens)
    with pytest.raises(cg.CacheGenError) as e:
        p.check()
    assert e.value.status == code
    assert np.array_equal(t.cpu().numpy(), table)
    assert p.lens.tolist() == lens and p.free_count.tolist() == [nfree]
    assert p.cu.tolist() == [0] * 4 and set(p.slots.tolist()) == {-1}


def test_grow_pages_reports_page_ids_outside_the_cache():
    p = cg.grow_pages(_ints([[99, -1], [1, -1]]), _ints([5, 5]), _ints([1, 1]), _ints([3]),
                      _ints([1]), 16, 2, num_pages=4)
    assert p.slots.tolist() == [-1, 16 + 5]
    with pytest.raises(cg.CacheGenError) as e:
        p.check()
    assert e.value.status == cg.CG_ERR_CORRUPT


def test_grow_pages_in_place_in_a_graph():
    """A captured step that advances lengths, tables and the free list in place."""
    page, n, steps = 16, 5, 40
    lens, free, nfree = _ints([0, 15, 16, 3, 31]), _ints(range(100)), _ints([100])
    table = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
    table[1, 0], table[2, 0], table[3, 0], table[4, 0], table[4, 1] = 100, 101, 102, 103, 104
    counts = _ints([1, 1, 0, 2, 1])
    plan = cg.PagePlan(torch.empty(8, dtype=torch.int32, device="cuda"),
                       torch.empty(n + 1, dtype=torch.int32, device="cuda"), lens, nfree,
                       torch.empty(16, dtype=torch.uint8, device="cuda"))
    wt, wl, wf = table.cpu().numpy(), lens.tolist(), 100
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        cg.grow_pages(table, lens, counts, free, nfree, page, 8, out=plan)
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        wt, ws, wf = _grow_ref(wt, wl, counts.tolist(), np.arange(100), wf, page, 8)
        wl = [a + b for a, b in zip(wl, counts.tolist())]
        assert plan.slots.tolist() == ws and lens.tolist() == wl and nfree.tolist() == [wf]
        assert np.array_equal(table.cpu().numpy(), wt)


# --------------------------------------------------------------- attention

def _batch(rng, nq, nkv, page, spare=3):
    """Block table and page count for requests of nkv tokens."""
    held = [-(-m // page) for m in nkv]
    pages = sum(held) + spare
    ids = rng.permutation(pages)
    table = np.full((len(nkv), max(max(held), 1) + 1), -1, np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = ids[at:at + h]
        at += h
    return table, pages


def _filled(rng, nkv, table, pages, page, heads, dim, group, layers=1, layer=0, scale=1.0, vscale=1.0):
    """A cache whose other places hold bytes that are no numbers."""
    want, got = _pair(layers, pages, page, heads, dim, group, fill=0xFF)
    for r, m in enumerate(nkv):
        x = np.arange(m)
        slots = table[r][x // page] * page + x % page
        k = ref.bf16_round(_rand(rng, m, heads, dim) * np.exp(0.7 * rng.standard_normal((heads, dim))) * scale)
        want.store(layer, k, ref.bf16_round((_rand(rng, m, heads, dim) + 0.5) * np.float32(vscale)), slots)
    _copy(want, got)
    return want, got


def _check_attention(out, want, tol):
    out = _np(out).astype(np.float64)
    worst = np.abs(out - want) - tol
    assert np.isfinite(out).all() and (worst <= 0).all(), \
        (float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))


def _run(rng, nq, nkv, heads, ratio, dim, group, page, window=0, sinks=0, scale=None, most=None,
         kscale=1.0, qscale=1.0, vscale=1.0):
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group, scale=kscale, vscale=vscale)
    cu = np.concatenate([[0], np.cumsum(nq)])
    T = int(cu[-1])
    q = _rand(rng, T + 2, heads * ratio, dim, scale=qscale)
    out = torch.full((T + 2, heads * ratio, dim), 77.0, dtype=torch.bfloat16, device="cuda")
    got.attention(_dev(q), _ints(cu), _ints(nkv), _ints(table), window=window, sinks=sinks,
                  scale=scale, max_q_len=most, out=out)
    got.check()
    assert bool((out[T:] == 77.0).all())     # rows behind the last request
    o, tol = ref.attention(want, 0, q[:T], cu, nkv, table, window, sinks,
                           dim ** -0.5 if scale is None else scale)
    _check_attention(out[:T], o, tol)
    return out


@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("heads,ratio,page", [(2, 1, 16), (1, 4, 48), (3, 7, 32), (1, 16, 64), (1, 24, 16)])
def test_attention_of_single_tokens(dim, group, heads, ratio, page):
    nkv = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257, 700]
    _run(np.random.default_rng(ratio + group), [1] * len(nkv), nkv, heads, ratio, dim, group, page, most=1)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 4), (17, 37), (100, 16), (1000, 4), (64, 0)])
@pytest.mark.parametrize("nq", [1, 3])
def test_attention_under_a_window(window, sinks, nq):
    nkv = [3, 15, 16, 17, 40, 90, 128, 129, 333, 800]
    _run(np.random.default_rng(window), [nq] * len(nkv), nkv, 2, 4, 128, 32, 16, window, sinks, most=nq)


@pytest.mark.parametrize("dim,group", FORMATS)
@pytest.mark.parametrize("heads,ratio", [(2, 1), (1, 3), (2, 4)])
def test_attention_of_prompts(dim, group, heads, ratio):
    nq = [200, 1, 65, 0, 129, 33]
    nkv = [200, 300, 100, 50, 400, 33]
    _run(np.random.default_rng(dim + ratio), nq, nkv, heads, ratio, dim, group, 16)


@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (64, 70), (200, 4), (128, 0)])
def test_attention_of_prompts_under_a_window(window, sinks):
    nq = [260, 1, 70, 100]
    nkv = [260, 500, 330, 900]
    _run(np.random.default_rng(window), nq, nkv, 1, 4, 128, 128, 32, window, sinks)


@pytest.mark.parametrize("nq", [1, 2, 4, 5, 8, 9, 16, 17, 31])
def test_attention_of_drafts(nq):
    nkv = [nq, 40, 170, 513]
    _run(np.random.default_rng(nq), [nq] * 4, nkv, 2, 4, 128, 64, 16, most=nq)


def test_attention_mixes_every_kind_of_request():
    nq = [1, 0, 7, 150, 1, 0, 16, 1, 300]
    nkv = [600, 0, 7, 150, 0, 20, 100, 1, 350]      # a row without any token, requests without rows
    _run(np.random.default_rng(1), nq, nkv, 2, 4, 128, 32, 16)
    _run(np.random.default_rng(2), nq, nkv, 3, 2, 64, 64, 48, window=33, sinks=2)


def test_attention_rows_before_the_first_token_are_zero():
    """More rows than cached tokens: the first rows stand before position 0."""
    out = _run(np.random.default_rng(3), [5, 40, 3], [3, 10, 0], 1, 2, 64, 32, 16)
    assert not _np(out)[:2].any() and not _np(out)[5:35].any() and not _np(out)[45:48].any()


@pytest.mark.parametrize("nq", [1, 90])
@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
def test_attention_scales(scale, nq):
    _run(np.random.default_rng(4), [nq, nq], [90, 111], 1, 4, 128, 32, 16, scale=scale)


@pytest.mark.parametrize("nq", [1, 80])
@pytest.mark.parametrize("kscale,qscale", [(1e-30, 1.0), (1e4, 1e-4), (1e-4, 1e4), (1e30, 1e-30)])
def test_attention_of_large_and_small_values(kscale, qscale, nq):
    _run(np.random.default_rng(5), [nq, nq], [80, 300], 1, 4, 128, 64, 16, kscale=kscale, qscale=qscale)


@pytest.mark.parametrize("nq", [1, 80])
@pytest.mark.parametrize("power", [-100, 5, 20, 90])
def test_attention_of_large_and_small_values_of_v(power, nq):
    _run(np.random.default_rng(14), [nq, nq], [90, 700], 1, 4, 128, 32, 16, vscale=2.0 ** power)


def test_attention_layers_strides_and_other_streams():
    rng = np.random.default_rng(6)
    heads, ratio, dim, group, page = 2, 4, 128, 32, 16
    nq, nkv = [1, 3, 100], [70, 40, 180]
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group, layers=3, layer=2)
    cu = np.concatenate([[0], np.cumsum(nq)])
    T, qh = int(cu[-1]), heads * ratio
    wide = _rand(rng, T, qh + 2 * heads, dim)          # q inside a fused projection
    w = _dev(wide)
    o, tol = ref.attention(want, 2, wide[:, :qh], cu, nkv, table, 0, 0, dim ** -0.5)
    tabs = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    tabs[:, :table.shape[1]] = _ints(table)
    tab = tabs[:, :table.shape[1]]                     # rows of a wider table
    outs = torch.zeros(qh, T, dim, dtype=torch.bfloat16, device="cuda")
    got.attention(w[:, :qh], _ints(cu), _ints(nkv), tab, layer=2, out=outs.transpose(0, 1))
    _check_attention(outs.transpose(0, 1), o, tol)
    args = w[:, :qh], _ints(cu), _ints(nkv), tab
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    res = [got.attention(*args, layer=2, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    for r in res:
        assert torch.equal(r, outs.transpose(0, 1))    # the same bits every time
    got.check()


def test_attention_does_not_read_pages_that_have_left_the_window():
    rng = np.random.default_rng(7)
    nkv, page, window, sinks = [333, 800], 16, 50, 4
    for nq in ([1, 1], [3, 2], [70, 90]):
        table, pages = _batch(rng, nq, nkv, page)
        want, got = _filled(rng, nkv, table, pages, page, 1, 128, 32)
        for r in range(2):
            first = nkv[r] - nq[r] + 1 - window           # the first row's window
            table[r, 1:first // page] = -1                # page 0 holds the sinks
        cu = np.concatenate([[0], np.cumsum(nq)])
        q = _rand(rng, int(cu[-1]), 4, 128)
        out = got.attention(_dev(q), _ints(cu), _ints(nkv), _ints(table), window=window, sinks=sinks)
        got.check()
        _check_attention(out, *ref.attention(want, 0, q, cu, nkv, table, window, sinks, 128 ** -0.5))


@pytest.mark.parametrize("nq", [1, 80])
def test_attention_reports_bad_pages_and_lengths(nq):
    rng = np.random.default_rng(8)
    nkv, page = [100, 90], 16
    table, pages = _batch(rng, [nq] * 2, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, 1, 64, 32)
    cu = np.array([0, nq, 2 * nq])
    q = _rand(rng, 2 * nq, 2, 64)

    def call(cu=cu, nkv=nkv, table=table, most=None):
        out = torch.full((2 * nq, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        got.attention(_dev(q), _ints(cu), _ints(nkv), _ints(table), max_q_len=most, out=out)
        with pytest.raises(cg.CacheGenError) as e:
            got.check()
        return out, e.value.status

    o, tol = ref.attention(want, 0, q, cu, nkv, table, 0, 0, 64 ** -0.5)
    for page_id in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[0, 2] = page_id                       # request 0 loses tokens 32..47
        out, st = call(table=t)
        assert st == cg.CG_ERR_CORRUPT
        _check_attention(out[nq:], o[nq:], tol[nq:])
        assert torch.isfinite(out.float()).all()
    for lens in ([-1, 90], [2 ** 31 - 1, 90], [table.shape[1] * page + 1, 90]):
        out, st = call(nkv=lens)
        assert st == cg.CG_ERR_CORRUPT and bool((out[:nq] == 5.0).all())
        _check_attention(out[nq:], o[nq:], tol[nq:])
    out, st = call(cu=np.array([-1, nq, 2 * nq]))
    assert st == cg.CG_ERR_CORRUPT
    _check_attention(out[nq:], o[nq:], tol[nq:])
    out, st = call(cu=np.array([0, nq, 2 * nq + 1]))
    assert st == cg.CG_ERR_CORRUPT and bool((out[nq:] == 5.0).all())
    _check_attention(out[:nq], o[:nq], tol[:nq])
    out, st = call(cu=np.array([nq, 0, 2 * nq]))
    assert st == cg.CG_ERR_CORRUPT
    if nq > 1:
        out, st = call(most=nq - 1)
        assert st == cg.CG_ERR_INVALID_ARG and bool((out == 5.0).all())


def test_attention_without_rows_or_requests():
    _, got = _pair(1, 1, 16, 1, 64, 32)
    out = got.attention(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), _ints([0, 0]),
                        _ints([5]), _ints([[0]]))
    assert out.shape == (0, 4, 64)
    keep = torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    got.attention(keep, _ints([0]), _ints([]), torch.empty(0, 3, dtype=torch.int32, device="cuda"), out=keep)
    got.attention(torch.ones_like(keep), _ints([0, 0]), _ints([5]), _ints([[0]]), out=keep)
    assert bool((keep == 2.0).all())
    got.check()


@pytest.mark.parametrize("n", [32, 33, 128, 129, 700, 8192])
def test_attention_of_many_requests(n):
    """Schedules within a warp, within a block and in two passes."""
    rng = np.random.default_rng(n)
    nkv = rng.integers(0, 60 if n < 1000 else 20, n)
    nq = rng.integers(0, 3, n)
    _run(rng, nq.tolist(), nkv.tolist(), 1, 2, 64, 64, 16, most=2)
    _run(rng, nq.tolist(), nkv.tolist(), 2, 1, 128, 128, 16, window=21, sinks=1)


@pytest.mark.parametrize("n", [31, 33, 140])
def test_attention_of_many_requests_with_many_rows(n):
    """Units of both kernels side by side, more of them than blocks."""
    rng = np.random.default_rng(n)
    nq = rng.choice([0, 1, 30, 40, 130], n, p=[0.1, 0.2, 0.3, 0.3, 0.1])
    nkv = nq + rng.integers(0, 50, n)
    _run(rng, nq.tolist(), nkv.tolist(), 2, 2, 64, 32, 16)


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32)])
@pytest.mark.parametrize("nq,window,sinks", [(13, 0, 0), (33, 0, 0), (64, 0, 0), (65, 700, 9), (13, 1000, 0)])
def test_attention_of_few_units_is_cut_along_the_tokens(dim, group, nq, window, sinks):
    """One and two row tiles of long requests: pieces, joined by the second kernel."""
    _run(np.random.default_rng(nq), [nq, nq], [3100, 2055], 1, 4, dim, group, 32, window, sinks, most=nq)


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_attention_keeps_a_row_that_is_not_finite_to_itself(bad, nq):
    rng = np.random.default_rng(11)
    nkv, page, heads, ratio, dim = [75, 200], 16, 1, 4, 128
    table, pages = _batch(rng, [nq, nq], nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, 32)
    cu = np.array([0, nq, 2 * nq])
    q = _rand(rng, 2 * nq, heads * ratio, dim)
    o, tol = ref.attention(want, 0, q, cu, nkv, table, 0, 0, dim ** -0.5)
    q[nq, 2, 7] = bad
    out = got.attention(_dev(q), _ints(cu), _ints(nkv), _ints(table))
    keep = np.ones(q.shape[:2], bool)
    keep[nq, 2] = False
    assert torch.isnan(out[nq, 2].float()).all()
    _check_attention(out[torch.from_numpy(keep).cuda()], o[keep], tol[keep])
    got.check()


def test_attention_graphs_and_streams_side_by_side():
    """Two captured graphs and eager calls, on three streams at once, prompts and single tokens: the
    same bits as alone. Lengths change between replays."""
    rng = np.random.default_rng(12)
    heads, ratio, dim, group, page = 2, 4, 128, 64, 16
    nq, nkv = [1, 2, 70, 200, 13], [900, 40, 300, 200, 2500]
    table, pages = _batch(rng, nq, nkv, page)
    want, got = _filled(rng, nkv, table, pages, page, heads, dim, group)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q, tab, cu_t = _dev(_rand(rng, int(cu[-1]), heads * ratio, dim)), _ints(table), _ints(cu)
    shorter = [m - d for m, d in zip(nkv, [300, 3, 41, 0, 1000])]
    alone = [got.attention(q, cu_t, _ints(l), tab) for l in (nkv, shorter)]
    _check_attention(alone[1], *ref.attention(want, 0, _np(q), cu, shorter, table, 0, 0, dim ** -0.5))
    lens = [_ints(nkv), _ints(nkv)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            outs.append(got.attention(q, cu_t, lens[i], tab))
        graphs.append(g)
    for turn in range(6):
        lens[turn % 2].copy_(_ints(shorter if turn < 3 else nkv))
        now = [torch.equal(l.cpu(), _ints(nkv).cpu()) for l in lens]
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        eager = got.attention(q, cu_t, lens[0], tab, stream=streams[2])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], alone[0 if now[i] else 1])
        assert torch.equal(eager, outs[0])
    got.check()


def test_offsets_past_32_bits():
    """A layer of 5 GB whose pages in use lie at its end: the same results as in a small cache."""
    rng = np.random.default_rng(13)
    heads, ratio, dim, group, page, pages = 8, 2, 128, 32, 1024, 4000
    big = cg.Int4Cache(1, pages, page, heads, dim, group,
                       data=torch.empty(pages * page // 16 * heads * 2560, dtype=torch.uint8, device="cuda"))
    small = cg.Int4Cache(1, 5, page, heads, dim, group)
    n = 3 * page + 77
    k, v = _dev(_rand(rng, n, heads, dim)), _dev(_rand(rng, n, heads, dim))
    ids = {small: [2, 0, 4, 1], big: [3999, 3, 3997, 3998]}
    x, got = np.arange(n), {}
    nq = [1, 40, 3]
    cu, lens = _ints([0, 1, 41, 44]), _ints([n, n - 5, 2 * page + 1])
    q = _dev(_rand(rng, 44, heads * ratio, dim))
    for c, page_ids in ids.items():
        slots = _ints(np.array(page_ids)[x // page] * page + x % page)
        c.store(k, v, slots)
        table = _ints([page_ids] * 3)
        got[c] = c.load(slots) + (c.attention(q, cu, lens, table, max_q_len=max(nq)),)
        c.check()
    for a, b in zip(got[small], got[big]):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- together

def test_a_restored_cache_is_attended_and_grown():
    """Codec.decode -> store -> decode steps (grow, store, attention) captured
    in a graph and replayed -> load -> Codec.encode, as a serving loop runs."""
    name = "mistral7b_t1k"
    p = synthetic.WORKLOADS[name]
    L, H, D, T0, page, steps, ratio = 3, p["H"], p["D"], 70, 16, 20, 4
    rng = np.random.default_rng(9)
    kv_bits = synthetic.generate(name, num_tokens=T0)[:L]
    kv = torch.from_numpy(kv_bits.view(np.int16)).view(torch.bfloat16).reshape(L, 2, T0, H, D).cuda()
    codec = cg.Codec(L, T0, H, D, 256)
    back = codec.decode(codec.encode(kv))
    pages = 24
    want, got = _pair(L, pages, page, H, D, 32)
    free, nfree = _ints(rng.permutation(pages)), _ints([pages])
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    lens = _ints([0, 0])
    plan = cg.grow_pages(table, lens, _ints([T0, 0]), free, nfree, page, T0, num_pages=pages)
    plan.check()
    got.store(back[:, 0], back[:, 1], plan.slots)
    for l in range(L):
        want.store(l, _np(back[l, 0]), _np(back[l, 1]), plan.slots.tolist())
    _same_bytes(want, got)
    # one captured step: both requests get a token (the batch is padded to 3 rows)
    lens, nfree = plan.lens, plan.free_count
    step = cg.PagePlan(torch.empty(3, dtype=torch.int32, device="cuda"),
                       torch.empty(3, dtype=torch.int32, device="cuda"), lens, nfree,
                       torch.empty(16, dtype=torch.uint8, device="cuda"))
    ones = _ints([1, 1])
    k = torch.zeros(L, 3, H, D, dtype=torch.bfloat16, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros(L, 3, H * ratio, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        cg.grow_pages(table, lens, ones, free, nfree, page, 3, out=step)
        for l in range(L):
            got.store(k[l], v[l], step.slots, layer=l)
            got.attention(q[l], step.cu, lens, table, layer=l, window=40, sinks=4, max_q_len=1, out=out[l])
    for i in range(steps):
        kn, vn, qn = _rand(rng, L, 3, H, D), _rand(rng, L, 3, H, D), _rand(rng, L, 3, H * ratio, D)
        k.copy_(_dev(kn)), v.copy_(_dev(vn)), q.copy_(_dev(qn))
        graph.replay()
        torch.cuda.synchronize()
        step.check()
        assert lens.tolist() == [T0 + i + 1, i + 1] and step.slots.tolist()[2] == -1
        for l in range(L):
            want.store(l, kn[l], vn[l], step.slots.tolist())
            o, tol = ref.attention(want, l, qn[l][:2], [0, 1, 2], lens.tolist(), table.cpu().numpy(), 40, 4, D ** -0.5)
            _check_attention(out[l, :2], o, tol)
    _same_bytes(want, got)
    got.check()
    # swap request 0 out again
    n = T0 + steps
    pos = torch.arange(n, device="cuda")
    slots = (table[0, pos // page] * page + pos % page).to(torch.int32)
    blob = torch.empty(L, 2, n, H, D, dtype=torch.bfloat16, device="cuda")
    got.load(slots, layers=L, k_out=blob[:, 0], v_out=blob[:, 1])
    c2 = cg.Codec(L, n, H, D, 256)
    again = c2.decode(c2.encode(blob))
    step64 = blob.float().abs().amax((3, 4), keepdim=True) / 7      # half a step of the 16-bin layers
    assert bool(((again.float() - blob.float()).abs() <= step64).all())


@pytest.mark.parametrize("dim,group", FORMATS)
def test_load_rounds_to_fp32_and_then_to_bf16(dim, group):
    """|lo| so small that fp32 drops it next to s n, which lies halfway between two bf16 values
    for some codes: the format's value is then the even one, not the one on lo's side."""
    top = 1 + np.arange(128) / 128                        # a binade of bf16: every mantissa of s
    rows = np.arange(group) % 16 / 15 * top[:, None, None]
    rows = np.tile(rows.astype(np.float32), (1, 1, dim // group))
    lo = ref.bf16_round(np.float32([-2.0 ** -30, 2.0 ** -30, -1.5 * 2.0 ** -40, 2.0 ** -22]))[np.arange(128) % 4]
    rows[:, :, ::group] = lo[:, None, None]
    rows[:, :, 16::group] = np.maximum(lo, rows[:, 0, 1])[:, None, None]
    rows = ref.bf16_round(rows)
    back = rows[::-1].copy()
    for slots in (np.arange(128), np.random.default_rng(group).permutation(128)):
        want, got = _pair(1, 8, 16, 1, dim, group)
        got.store(_dev(rows), _dev(back), _ints(slots))
        want.store(0, rows, back, slots)
        _same_bytes(want, got)
        k, v, _ = want.values(0, slots)
        for w, l in zip((k, v), got.load(_ints(slots))):
            assert np.array_equal(ref.bits(_np(l)), ref.bits(ref.bf16_round(w.astype(np.float32))))
    # where one rounding would give others: fp32 drops lo and s n is halfway
    half = (np.float32(k).view(np.uint32) & 0xFFFF) == 0x8000
    assert (half & (np.float32(k).astype(np.float64) != k)).sum() > 50


def test_check_keeps_an_error_that_comes_while_it_reads(monkeypatch):
    """A store on another stream meets an error after check() has read the first one."""
    _, got = _pair(1, 2, 16, 1, 64, 64)
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    got.store(k, k, _ints([99]))
    read, other = cg.cg_last_device_error, torch.cuda.Stream()
    bad = torch.full_like(k, float("nan"))
    slot = _ints([3])

    def read_and_then_store(*args):
        st = read(*args)
        got.store(bad, k, slot, stream=other)
        other.synchronize()
        return st

    with monkeypatch.context() as m:
        m.setattr(cg, "cg_last_device_error", read_and_then_store)
        with pytest.raises(cg.CacheGenError) as e:
            got.check()
        assert e.value.status == cg.CG_ERR_CORRUPT
    with pytest.raises(cg.CacheGenError) as e:
        got.check()
    assert e.value.status == cg.CG_ERR_NONFINITE
    got.check()


def test_inputs_may_be_dropped_while_another_stream_reads_them():
    """Calls with stream= that wait behind other work there: memory of inputs that the caller has
    dropped is not handed out again before they have run."""
    rng = np.random.default_rng(15)
    n, heads, dim, page = 4096, 2, 128, 64
    got, other = cg.Int4Cache(1, n // page, page, heads, dim, 32), torch.cuda.Stream()
    k, v, q = (_dev(_rand(rng, n, heads * m, dim)) for m in (1, 1, 4))
    slots, table, lens = _ints(rng.permutation(n)), _ints([rng.permutation(n // page)] * n), _ints(rng.integers(1, n, n))
    cu = _ints(np.arange(n + 1))

    def pages(stream=None, args=None):
        a = args or make()
        return cg.grow_pages(*a, 16, 70000, stream=stream)

    def make():
        return (torch.full((n, 300), -1, dtype=torch.int32, device="cuda"), torch.zeros_like(lens), lens // 256,
                torch.arange(n * 2, dtype=torch.int32, device="cuda").flip(0), _ints([n * 2]))

    got.store(k, v, slots)
    want = got.load(slots) + (got.attention(q, cu, lens, table, max_q_len=1),)
    plan = pages()
    bytes_ = got.data.clone()
    torch.cuda.synchronize()

    def later(call, *args, **kw):
        """call on copies of args that are dropped at once, their memory taken by other tensors."""
        copies = [a.clone() for a in args]
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            torch.cuda._sleep(100_000_000)
        res = call(*copies, stream=other, **kw)
        copies.clear()
        junk = [torch.full_like(a, 3) for _ in range(3) for a in args]
        torch.cuda.synchronize()
        del junk
        return res

    assert torch.equal(later(got.attention, q, cu, lens, table, max_q_len=1), want[2])
    for a, b in zip(later(got.load, slots), want):
        assert torch.equal(a, b)
    got.data.zero_()
    later(got.store, k, v, slots)
    assert torch.equal(got.data, bytes_)
    p = later(lambda *a, stream: pages(stream, a), *make())
    assert p.slots.tolist() == plan.slots.tolist() and p.cu.tolist() == plan.cu.tolist()
    got.check(), p.check()


@pytest.mark.parametrize("n", [40, 3000])
def test_grow_pages_reports_the_same_of_several_errors(n):
    """Whichever thread meets its error first: the greatest code."""
    rng = np.random.default_rng(n)
    for wrong, code in (("negative, narrow", cg.CG_ERR_CAPACITY), ("negative, list", cg.CG_ERR_CORRUPT),
                        ("negative, pages", cg.CG_ERR_CAPACITY), ("narrow, list", cg.CG_ERR_CORRUPT),
                        ("pages, list", cg.CG_ERR_CORRUPT), ("negative, narrow, pages, list", cg.CG_ERR_CORRUPT)):
        for _ in range(4):
            at = rng.permutation(n)
            lens, counts, nfree = np.full(n, 5), np.full(n, 1), 8
            if "negative" in wrong:
                lens[at[0]] = -1
            if "narrow" in wrong:
                lens[at[1]] = 100
            if "pages" in wrong:
                counts[at[2]], nfree = 40, 1
            if "list" in wrong:
                nfree = 9 if "pages" not in wrong else -1
            p = cg.grow_pages(_ints(np.zeros((n, 4))), _ints(lens), _ints(counts), _ints(range(8)), _ints([nfree]), 16,
                              n + 40)
            with pytest.raises(cg.CacheGenError) as e:
                p.check()
            assert e.value.status == code, wrong


def test_numbers_past_32_bits_are_refused_and_not_cut_off():
    _, got = _pair(1, 2, 16, 1, 64, 64)
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    one, table = _ints([1]), _ints([[0]])
    for call in (lambda: got.store(k, k, one, layer=2 ** 32), lambda: got.load(one, layer=2 ** 32),
                 lambda: got.load(one, layers=2 ** 32 + 1), lambda: got.attention(k, _ints([0, 1]), one, table, layer=2 ** 32),
                 lambda: got.attention(k, _ints([0, 1]), one, table, window=2 ** 40),
                 lambda: cg.grow_pages(table, one, one, one, one, 2 ** 33, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(cg.CacheGenError) as e:      # fp32's infinity
        got.attention(k, _ints([0, 1]), one, table, scale=1e39)
    assert e.value.status == cg.CG_ERR_INVALID_ARG
    assert not got.data.any()
    got.check()
