"""Host-side checks of eviction from the 4-bit paged cache and of attention with shared tokens
(no GPU needed): every refusal of the C calls and of their binding, which come back before
any device work is enqueued, and the numpy forms that the GPU tests go by."""
import ctypes as ct

import numpy as np
import pytest
import torch

import evict_ref as evict
import int4_ref as ref
from kv_cache_compression_03_gb300 import cachegen as cg

from test_int4_host import BAD_POINTERS, BAD_SHAPES, FAKE, _args, _cache

INV, UNS = cg.CG_ERR_INVALID_ARG, cg.CG_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return cg.load()


def _make(kind, d, kw):
    assert set(kw) <= set(d)
    return kind(**{**d, **kw})


def test_shared_attention_refusals(lib):
    n = ct.c_size_t(0)

    def need(cache=None, args=None, shared=32):
        return lib.cg_int4_attention_shared_workspace(ct.byref(cache or _cache()), ct.byref(args or _args()), shared,
                                                      ct.byref(n))

    def go(cache=None, args=None, shared=32, layer=0, ws=FAKE, size=1 << 40):
        return lib.cg_int4_attention_shared(ct.byref(cache or _cache()), layer, ct.byref(args or _args()), shared, ws,
                                            size, None)

    assert need() == cg.CG_OK and n.value >= 3 * 16 * 130 * 4
    most = n.value
    for kw, code in BAD_SHAPES:
        assert need(_cache(**kw)) == code and go(_cache(**kw)) == code, kw
    for kw, code in BAD_POINTERS:
        assert go(_cache(**kw)) == code, kw
    for shared in (-16, 8, 33, 9 * 16, 1 << 30):
        assert need(shared=shared) == INV and go(shared=shared) == INV, shared
    assert need(args=_args(window=5)) == INV and go(args=_args(window=5)) == INV
    assert need(args=_args(tokens=1 << 27)) == UNS
    for kw in (dict(q=0), dict(out=0), dict(cu_q=0), dict(kv_lens=0), dict(block_table=0), dict(q=FAKE + 8),
               dict(q_token_stride=4), dict(out_head_stride=1)):
        assert go(args=_args(**kw)) == INV, kw
    assert go(layer=-1) == INV and go(layer=2) == INV and go(ws=FAKE + 16) == INV
    assert go(size=most - 1) == cg.CG_ERR_CAPACITY and go(ws=None) == cg.CG_ERR_CAPACITY
    assert lib.cg_int4_attention_shared_workspace(None, ct.byref(_args()), 32, ct.byref(n)) == INV
    # without shared tokens it is the other call
    assert need(shared=0) == cg.CG_OK
    assert lib.cg_int4_attention_workspace(ct.byref(_cache()), ct.byref(_args()), ct.byref(ct.c_size_t(0))) == cg.CG_OK
    assert go(args=_args(tokens=0, q=0, out=0)) == cg.CG_OK
    assert go(args=_args(requests=0, cu_q=0, kv_lens=0)) == cg.CG_OK


def _weights(**kw):
    return _make(cg.cg_token_weights, dict(in_=FAKE, out=FAKE, in_request_stride=512, in_head_stride=128,
                                           out_request_stride=512, out_head_stride=128, width=128), kw)


def test_weigh_refusals(lib):
    n = ct.c_size_t(0)

    def need(cache=None, args=None, w=None):
        return lib.cg_int4_weigh_workspace(ct.byref(cache or _cache()), ct.byref(args or _args()),
                                           ct.byref(w or _weights()), ct.byref(n))

    def go(cache=None, args=None, w=None, layer=0, ws=FAKE, size=1 << 40):
        return lib.cg_int4_weigh(ct.byref(cache or _cache()), layer, ct.byref(args or _args()),
                                 ct.byref(w or _weights()), ws, size, None)

    assert need() == cg.CG_OK and n.value > 0
    most = n.value
    for kw, code in BAD_SHAPES:
        assert need(_cache(**kw)) == code and go(_cache(**kw)) == code, kw
    for kw, code in BAD_POINTERS:
        assert go(_cache(**kw)) == code, kw
    for kw, code in ((dict(requests=-1), INV), (dict(tokens=-1), INV), (dict(q_heads=6), INV), (dict(window=-1), INV),
                     (dict(scale=float("nan")), INV), (dict(requests=8193), UNS), (dict(tokens=1 << 27), UNS)):
        assert need(args=_args(**kw)) == code and go(args=_args(**kw)) == code, kw
    for kw in (dict(width=-1), dict(out_request_stride=-1), dict(out_head_stride=-4), dict(in_request_stride=-1),
               dict(in_head_stride=-1)):
        assert need(w=_weights(**kw)) == INV and go(w=_weights(**kw)) == INV, kw
    for kw in (dict(out=0), dict(out=FAKE + 2), dict(in_=FAKE + 1), dict(in_head_stride=64), dict(in_request_stride=8)):
        assert go(w=_weights(**kw)) == INV, kw
    for kw in (dict(q=0), dict(cu_q=0), dict(kv_lens=0), dict(block_table=0), dict(q=FAKE + 8), dict(cu_q=FAKE + 1),
               dict(q_token_stride=4), dict(q_head_stride=-8)):
        assert go(args=_args(**kw)) == INV, kw
    assert go(layer=-1) == INV and go(layer=2) == INV and go(ws=FAKE + 16) == INV
    assert go(size=most - 1) == cg.CG_ERR_CAPACITY and go(ws=None) == cg.CG_ERR_CAPACITY
    for args in ((None, ct.byref(_args()), ct.byref(_weights())), (ct.byref(_cache()), None, ct.byref(_weights())),
                 (ct.byref(_cache()), ct.byref(_args()), None)):
        assert lib.cg_int4_weigh_workspace(*args, ct.byref(n)) == INV
    # nothing to do; out's strides in args are not looked at
    assert go(args=_args(requests=0, cu_q=0, kv_lens=0)) == cg.CG_OK
    assert go(args=_args(out=0, out_token_stride=3), size=0) == cg.CG_ERR_CAPACITY


def test_weigh_of_no_earlier_weights_into_rows_without_room(lib):
    """in and out are both none, and are not the same rows: in's strides are not looked at."""
    n = ct.c_size_t(0)
    w = _weights(in_=0, out=0, in_request_stride=0, in_head_stride=0, out_request_stride=4, out_head_stride=1, width=0)
    assert lib.cg_int4_weigh_workspace(ct.byref(_cache()), ct.byref(_args()), ct.byref(w), ct.byref(n)) == cg.CG_OK
    # all arguments are looked at before the workspace
    assert lib.cg_int4_weigh(ct.byref(_cache()), 0, ct.byref(_args()), ct.byref(w), None, 0, None) == cg.CG_ERR_CAPACITY
    w = _weights(in_=0, out=FAKE, in_request_stride=-1, in_head_stride=7)
    assert lib.cg_int4_weigh(ct.byref(_cache()), 0, ct.byref(_args()), ct.byref(w), None, 0, None) == cg.CG_ERR_CAPACITY


def _choice(**kw):
    return _make(cg.cg_token_choice, dict(weights=FAKE, layer_stride=4096, request_stride=1024, head_stride=256, layers=2,
                                          requests=3, heads=4, width=200, lens=FAKE, budget=50, recent=8, sinks=4,
                                          kept=FAKE, lens_out=FAKE, status=FAKE), kw)


def test_choose_refusals(lib):
    def go(**kw):
        return lib.cg_choose_tokens(ct.byref(_choice(**kw)), None)

    for kw in (dict(layers=-1), dict(requests=-1), dict(heads=-1), dict(width=-1), dict(budget=-1), dict(recent=-1),
               dict(sinks=-1), dict(recent=47), dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(layer_stride=-1),
               dict(request_stride=-1), dict(head_stride=-1), dict(weights=0), dict(lens=0), dict(kept=0),
               dict(lens_out=0), dict(status=0), dict(status=FAKE + 8), dict(weights=FAKE + 2), dict(lens=FAKE + 1),
               dict(kept=FAKE + 2), dict(lens_out=FAKE + 3)):
        assert go(**kw) == INV, kw
    for kw in (dict(requests=8193), dict(layers=1 << 30, requests=2), dict(layers=1 << 20, heads=1 << 20)):
        assert go(**kw) == UNS, kw
    assert lib.cg_choose_tokens(None, None) == INV


def _compaction(**kw):
    return _make(cg.cg_compaction, dict(kept=FAKE, kept_layer_stride=600, kept_request_stride=200, kept_head_stride=50,
                                        weights=FAKE, weights_layer_stride=2400, weights_request_stride=800,
                                        weights_head_stride=200, weights_width=128, budget=50, layers=2, requests=3,
                                        lens=FAKE, new_lens=FAKE, block_table=FAKE, table_stride=8, table_width=8), kw)


def test_compact_refusals(lib):
    def go(cache=None, layer=0, **kw):
        return lib.cg_int4_compact(ct.byref(cache or _cache()), layer, ct.byref(_compaction(**kw)), None)

    for kw, code in BAD_SHAPES + BAD_POINTERS:
        assert go(_cache(**kw)) == code, kw
    for kw in (dict(layers=-1), dict(requests=-1), dict(budget=-1), dict(table_width=-1), dict(table_stride=7),
               dict(kept_layer_stride=-1), dict(kept_request_stride=-1), dict(kept_head_stride=-1),
               dict(weights_width=-1), dict(weights_layer_stride=-1), dict(weights_request_stride=-1),
               dict(weights_head_stride=-1), dict(layers=3), dict(kept=0), dict(lens=0), dict(new_lens=0),
               dict(block_table=0), dict(kept=FAKE + 2), dict(weights=FAKE + 1), dict(lens=FAKE + 2),
               dict(new_lens=FAKE + 1), dict(block_table=FAKE + 2)):
        assert go(**kw) == INV, kw
    assert go(layer=-1) == INV and go(layer=1) == INV
    for kw in (dict(requests=8193), dict(table_width=1 << 27, table_stride=1 << 27)):
        assert go(**kw) == UNS, kw
    assert lib.cg_int4_compact(ct.byref(_cache()), 0, None, None) == INV
    assert go(layers=0, kept=0, lens=0) == cg.CG_OK and go(requests=0, new_lens=0) == cg.CG_OK


def _release(**kw):
    return _make(cg.cg_page_release, dict(block_table=FAKE, table_stride=8, table_width=8, requests=3, lens=FAKE,
                                          new_lens=FAKE, free_pages=FAKE, free_count=FAKE, free_capacity=20,
                                          num_pages=30, page_tokens=16, cu_out=FAKE, lens_out=FAKE,
                                          free_count_out=FAKE, status=FAKE), kw)


def test_release_refusals(lib):
    for kw in (dict(requests=-1), dict(table_width=-1), dict(table_stride=7), dict(free_capacity=-1), dict(num_pages=0),
               dict(page_tokens=0), dict(status=0), dict(status=FAKE + 4), dict(free_count=0), dict(cu_out=0),
               dict(free_count_out=0), dict(lens=0), dict(new_lens=0), dict(lens_out=0), dict(block_table=0),
               dict(free_pages=0), dict(block_table=FAKE + 1), dict(lens=FAKE + 2), dict(new_lens=FAKE + 2),
               dict(free_pages=FAKE + 1), dict(free_count=FAKE + 2), dict(cu_out=FAKE + 2), dict(lens_out=FAKE + 1),
               dict(free_count_out=FAKE + 3)):
        assert lib.cg_pages_release(ct.byref(_release(**kw)), None) == INV, kw
    for kw in (dict(page_tokens=20), dict(page_tokens=2048), dict(num_pages=1 << 27), dict(requests=8193)):
        assert lib.cg_pages_release(ct.byref(_release(**kw)), None) == UNS, kw
    assert lib.cg_pages_release(None, None) == INV


# ------------------------------------------------------------- the binding

CPU = torch.device("cpu")


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cg.release_pages(i[None].expand(2, 2).contiguous(), i, i, i, i[:1], 16)
    with pytest.raises(ValueError):
        cg.choose_tokens(torch.zeros(2, 1, 5), i, 3)


def test_binding_checks_weights():
    x = torch.zeros(3, 4, 50)
    for t in (x, x[:, 1:3], x[::2], x.transpose(0, 1), x[..., 3:40], x[:0], x[..., :0], x[..., ::2][..., :1]):
        cg._floats(t, CPU, tuple(t.shape), "x", True)
    same = x[:1].expand(3, 4, 50)
    cg._floats(same, CPU, (3, 4, 50), "x", False)
    overlap = torch.zeros(500).as_strided((3, 4, 50), (20, 50, 1))
    for bad, written in ((same, True), (overlap, True), (x.double(), False), (x.bfloat16(), False), (x[..., ::2], False),
                         (x.transpose(1, 2), False)):
        with pytest.raises(ValueError):
            cg._floats(bad, CPU, tuple(bad.shape), "x", written)
    with pytest.raises(ValueError):
        cg._floats(x[:2], CPU, (3, 4, 50), "x", False)
    with pytest.raises(ValueError):
        cg._floats(x, torch.device("cuda", 0), (3, 4, 50), "x", False)
    g = torch.zeros(3, 4, 50, requires_grad=True)
    with pytest.raises(ValueError, match="requires grad"):
        cg._floats(g * 2, CPU, (3, 4, 50), "x", False)
    cg._floats(g.detach(), CPU, (3, 4, 50), "x", True)


# ---------------------------------------------------------- the numpy forms

def test_numpy_choice():
    w = np.array([[[5, 1, 1, 3, 1, 9, 0, 2]]], np.float32)
    kept, new = evict.choose(w, [8], 5, 1, 1)
    assert kept.tolist() == [[[0, 1, 3, 5, 7]]] and new.tolist() == [5]
    kept, new = evict.choose(w, [4], 5, 1, 1)
    assert kept.tolist() == [[[0, 1, 2, 3, -1]]] and new.tolist() == [4]


def test_numpy_move_and_release():
    """What stays reads as before, at its new places."""
    rng = np.random.default_rng(0)
    cache = ref.Cache(1, 6, 16, 2, 64, 32)
    k = ref.bf16_round(rng.standard_normal((70, 2, 64)).astype(np.float32))
    table = np.array([[4, 1, 0, 5, 2]])
    slots = table[0][np.arange(70) // 16] * 16 + np.arange(70) % 16
    cache.store(0, k, -k, slots)
    kept = np.stack([np.sort(rng.permutation(70)[:33]) for _ in range(2)])[None, None]
    before = cache.values(0, slots)
    evict.compact(cache, 0, kept, [33], [70], table)
    after = cache.values(0, slots[:33])
    for h in range(2):
        for a, b in zip(after, before):
            assert np.array_equal(a[:, h], b[kept[0, 0, h], h])
    t, f, n, cu = evict.release(table, [70], [33], np.full(4, -7), 1, 16)
    assert t.tolist() == [[4, 1, 0, -1, -1]] and f.tolist() == [-7, 5, 2, -7] and n == 3 and cu.tolist() == [0, 2]
