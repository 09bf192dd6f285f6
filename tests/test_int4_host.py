"""Host-side checks of the 4-bit paged cache (no GPU needed): sizes, and
every refusal of the C calls and of their binding, which come back before any
device work is enqueued."""
import ctypes as ct

import pytest
import torch

from kv_cache_compression_03_gb300 import cachegen as cg

FAKE = 1 << 20   # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    return cg.load()


def _cache(**kw):
    d = dict(data=FAKE, status=FAKE, num_layers=2, num_pages=10, page_tokens=16, num_heads=4,
             head_size=128, group=32)
    d.update(kw)
    return cg.cg_int4_cache(*[d[n] for n, _ in cg.cg_int4_cache._fields_])


@pytest.mark.parametrize("D,G,blob", [(64, 32, 1280), (64, 64, 1152), (128, 32, 2560),
                                      (128, 64, 2304), (128, 128, 2176)])
def test_cache_bytes(lib, D, G, blob):
    n = ct.c_size_t(0)
    c = _cache(data=0, status=0, head_size=D, group=G, page_tokens=48)
    assert lib.cg_int4_cache_bytes(ct.byref(c), ct.byref(n)) == cg.CG_OK
    assert n.value == 2 * 10 * 4 * 3 * blob
    # more than 2^32 bytes
    c = _cache(data=0, status=0, num_layers=40, num_pages=60000, num_heads=8, head_size=D, group=G)
    assert lib.cg_int4_cache_bytes(ct.byref(c), ct.byref(n)) == cg.CG_OK
    assert n.value == 40 * 60000 * 8 * blob


BAD_SHAPES = [(dict(num_layers=0), cg.CG_ERR_INVALID_ARG), (dict(num_pages=-1), cg.CG_ERR_INVALID_ARG),
              (dict(num_heads=0), cg.CG_ERR_INVALID_ARG), (dict(page_tokens=0), cg.CG_ERR_INVALID_ARG),
              (dict(head_size=0), cg.CG_ERR_INVALID_ARG), (dict(group=0), cg.CG_ERR_INVALID_ARG),
              (dict(page_tokens=24), cg.CG_ERR_UNSUPPORTED), (dict(page_tokens=1040), cg.CG_ERR_UNSUPPORTED),
              (dict(head_size=96), cg.CG_ERR_UNSUPPORTED), (dict(group=16), cg.CG_ERR_UNSUPPORTED),
              (dict(head_size=64, group=128), cg.CG_ERR_UNSUPPORTED),
              (dict(num_pages=1 << 27), cg.CG_ERR_UNSUPPORTED),
              (dict(num_layers=1 << 15, num_pages=1 << 14), cg.CG_ERR_UNSUPPORTED),
              (dict(num_layers=1, num_pages=1, num_heads=1 << 22), cg.CG_ERR_UNSUPPORTED)]
BAD_POINTERS = [(dict(data=0), cg.CG_ERR_INVALID_ARG), (dict(data=FAKE + 128), cg.CG_ERR_INVALID_ARG),
                (dict(status=0), cg.CG_ERR_INVALID_ARG), (dict(status=FAKE + 8), cg.CG_ERR_INVALID_ARG)]


def _rows(**kw):
    d = dict(k=FAKE, v=FAKE, k_layer_stride=8192, k_token_stride=512, k_head_stride=128,
             v_layer_stride=8192, v_token_stride=512, v_head_stride=128)
    d.update(kw)
    return cg.cg_kv_rows(*[d[n] for n, _ in cg.cg_kv_rows._fields_])


@pytest.mark.parametrize("call", ["cg_int4_store", "cg_int4_load"])
def test_store_and_load_refusals(lib, call):
    f = getattr(lib, call)
    inv, uns = cg.CG_ERR_INVALID_ARG, cg.CG_ERR_UNSUPPORTED

    def go(cache=None, first=0, layers=1, rows=None, slots=FAKE, tokens=3):
        return f(ct.byref(cache or _cache()), first, layers, ct.byref(rows or _rows()), slots, tokens, None)

    for kw, code in BAD_SHAPES + BAD_POINTERS:
        assert go(_cache(**kw)) == code, kw
    assert f(None, 0, 1, ct.byref(_rows()), FAKE, 3, None) == inv
    assert f(ct.byref(_cache()), 0, 1, None, FAKE, 3, None) == inv
    for first, layers in ((-1, 1), (0, -1), (0, 3), (2, 1), (3, 0), (1, 2 ** 31 - 1)):
        assert go(first=first, layers=layers) == inv
    assert go(tokens=-1) == inv and go(slots=None) == inv and go(slots=FAKE + 2) == inv
    for kw in (dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(k_token_stride=4),
               dict(v_head_stride=-8), dict(k_layer_stride=12), dict(v_layer_stride=1)):
        assert go(rows=_rows(**kw)) == inv, kw
    assert go(tokens=1 << 31) == uns
    # nothing to do: no pointer is looked at
    assert go(layers=0) == cg.CG_OK and go(tokens=0, slots=None, rows=_rows(k=0, v=0)) == cg.CG_OK
    assert go(first=2, layers=0) == cg.CG_OK


def _batch(**kw):
    d = dict(block_table=FAKE, table_stride=8, table_width=8, requests=3, lens=FAKE, counts=FAKE,
             free_pages=FAKE, free_count=FAKE, free_capacity=10, num_pages=10, page_tokens=16,
             cu_out=FAKE, lens_out=FAKE, free_count_out=FAKE, slots_out=FAKE, tokens=5, status=FAKE)
    d.update(kw)
    return cg.cg_page_batch(*[d[n] for n, _ in cg.cg_page_batch._fields_])


def test_grow_refusals(lib):
    inv, uns = cg.CG_ERR_INVALID_ARG, cg.CG_ERR_UNSUPPORTED
    assert lib.cg_pages_grow(None, None) == inv
    for kw in (dict(requests=-1), dict(tokens=-1), dict(table_width=-1), dict(table_stride=7),
               dict(free_capacity=-1), dict(num_pages=0), dict(page_tokens=0), dict(status=0),
               dict(status=FAKE + 4), dict(free_count=0), dict(cu_out=0), dict(free_count_out=0),
               dict(lens=0), dict(counts=0), dict(lens_out=0), dict(block_table=0), dict(free_pages=0),
               dict(slots_out=0), dict(lens=FAKE + 1), dict(block_table=FAKE + 2), dict(slots_out=FAKE + 3)):
        assert lib.cg_pages_grow(ct.byref(_batch(**kw)), None) == inv, kw
    for kw in (dict(page_tokens=20), dict(page_tokens=2048), dict(num_pages=1 << 27),
               dict(requests=8193), dict(tokens=1 << 31)):
        assert lib.cg_pages_grow(ct.byref(_batch(**kw)), None) == uns, kw


def _args(**kw):
    d = dict(q=FAKE, q_token_stride=2048, q_head_stride=128, out=FAKE, out_token_stride=2048,
             out_head_stride=128, cu_q=FAKE, kv_lens=FAKE, block_table=FAKE, table_stride=8,
             table_width=8, requests=3, tokens=3, q_heads=16, max_q_len=0, window=0, sinks=0, scale=0.1)
    d.update(kw)
    return cg.cg_attention(*[d[n] for n, _ in cg.cg_attention._fields_])


def test_attention_refusals(lib):
    inv, uns = cg.CG_ERR_INVALID_ARG, cg.CG_ERR_UNSUPPORTED
    n = ct.c_size_t(0)

    def need(cache=None, args=None):
        return lib.cg_int4_attention_workspace(ct.byref(cache or _cache()), ct.byref(args or _args()), ct.byref(n))

    def go(cache=None, args=None, layer=0, ws=FAKE, size=1 << 40):
        return lib.cg_int4_attention(ct.byref(cache or _cache()), layer, ct.byref(args or _args()), ws, size, None)

    assert need() == cg.CG_OK
    for kw, code in BAD_SHAPES:
        assert need(_cache(**kw)) == code and go(_cache(**kw)) == code, kw
    for kw, code in BAD_POINTERS:
        assert go(_cache(**kw)) == code, kw
    sizes = [(dict(requests=-1), inv), (dict(tokens=-1), inv), (dict(q_heads=0), inv), (dict(q_heads=6), inv),
             (dict(max_q_len=-1), inv), (dict(window=-1), inv), (dict(sinks=-1), inv),
             (dict(table_width=-1), inv), (dict(table_stride=7), inv), (dict(scale=float("nan")), inv),
             (dict(scale=float("inf")), inv), (dict(requests=8193), uns),
             (dict(table_width=1 << 27, table_stride=1 << 27), uns), (dict(tokens=1 << 27), uns)]
    for kw, code in sizes:
        assert need(args=_args(**kw)) == code and go(args=_args(**kw)) == code, kw
    for kw in (dict(q=0), dict(out=0), dict(cu_q=0), dict(kv_lens=0), dict(block_table=0), dict(q=FAKE + 8),
               dict(out=FAKE + 2), dict(cu_q=FAKE + 1), dict(kv_lens=FAKE + 2), dict(block_table=FAKE + 1),
               dict(q_token_stride=4), dict(q_head_stride=-8), dict(out_token_stride=9), dict(out_head_stride=1)):
        assert go(args=_args(**kw)) == inv, kw
    assert go(layer=-1) == inv and go(layer=2) == inv and go(ws=FAKE + 16) == inv
    if n.value:
        assert go(size=n.value - 1) == cg.CG_ERR_CAPACITY
    assert lib.cg_int4_attention_workspace(None, ct.byref(_args()), ct.byref(n)) == inv
    assert lib.cg_int4_attention_workspace(ct.byref(_cache()), ct.byref(_args()), None) == inv
    # nothing to do
    assert go(args=_args(tokens=0, q=0, out=0)) == cg.CG_OK
    assert go(args=_args(requests=0, cu_q=0, kv_lens=0)) == cg.CG_OK


# ------------------------------------------------------------ the binding

CPU = torch.device("cpu")


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    with pytest.raises(ValueError):
        cg.Int4Cache(1, 2, 16, 1, 64, 32, data=torch.zeros(2 * 1280, dtype=torch.uint8))
    with pytest.raises(cg.CacheGenError) as e:
        cg.Int4Cache(1, 2, 16, 1, 80, 32, device="cpu")
    assert e.value.status == cg.CG_ERR_UNSUPPORTED
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cg.grow_pages(i[None].expand(2, 2).contiguous(), i, i, i, i[:1], 16, 2)


def test_binding_checks_integer_tensors():
    t = torch.zeros(4, dtype=torch.int32)
    cg._ints(t, CPU, (4,), "x")
    for bad, shape in ((t, (3,)), (t.long(), (4,)), (t[::2], (2,)), (t[None], (4,)), ([0] * 4, (4,))):
        with pytest.raises(ValueError):
            cg._ints(bad, CPU, shape, "x")
    with pytest.raises(ValueError):
        cg._ints(t, torch.device("cuda", 0), (4,), "x")
    table = torch.zeros(3, 8, dtype=torch.int32)
    cg._table(table[:, :5], CPU, "x")
    cg._table(table[:, :0], CPU, "x")
    for bad in (table.t(), table.long(), table[0], table[:, ::2], table[:1].expand(3, 8)):
        with pytest.raises(ValueError):
            cg._table(bad, CPU, "x")


def test_binding_checks_rows():
    x = torch.zeros(5, 6, 64, dtype=torch.bfloat16)
    ok = [x, x[:, 1:3], x[::2], x.transpose(0, 1).contiguous().transpose(0, 1), x[:0], x[:, :, :64]]
    for t in ok:
        cg._bf16_rows(t, CPU, tuple(t.shape), "x", True)
    same = x[:1].expand(5, 6, 64)
    cg._bf16_rows(same, CPU, (5, 6, 64), "x", False)          # one row read for all
    with pytest.raises(ValueError):
        cg._bf16_rows(same, CPU, (5, 6, 64), "x", True)       # but not written
    overlap = torch.zeros(2000, dtype=torch.bfloat16).as_strided((5, 6, 64), (32, 64, 1))
    with pytest.raises(ValueError):
        cg._bf16_rows(overlap, CPU, (5, 6, 64), "x", True)
    wide = torch.zeros(5, 6, 68, dtype=torch.bfloat16)
    for bad in (x.float(), x.half(), x[:4], x.transpose(1, 2), wide[:, :, :64], wide[:, :, 4:],
                torch.zeros(5, 6, 128, dtype=torch.bfloat16)[:, :, ::2]):
        with pytest.raises(ValueError):
            cg._bf16_rows(bad, CPU, (5, 6, 64), "x", False)
    with pytest.raises(ValueError):
        cg._bf16_rows(x, torch.device("cuda", 0), (5, 6, 64), "x", False)


def test_attention_refuses_a_scale_whose_powers_of_two_overflow(lib):
    """Scores are taken times log2 e."""
    n = ct.c_size_t(0)
    for scale, code in ((3.0e38, cg.CG_ERR_INVALID_ARG), (-2.4e38, cg.CG_ERR_INVALID_ARG), (2.3e38, cg.CG_OK)):
        assert lib.cg_int4_attention_workspace(ct.byref(_cache()), ct.byref(_args(scale=scale)), ct.byref(n)) == code


def test_take_error_refusals(lib):
    f, inv = lib.cg_int4_take_error, cg.CG_ERR_INVALID_ARG
    for kw, code in BAD_SHAPES + BAD_POINTERS:
        assert f(ct.byref(_cache(**kw)), FAKE, None) == code, kw
    assert f(None, FAKE, None) == inv and f(ct.byref(_cache()), None, None) == inv
    assert f(ct.byref(_cache()), FAKE + 8, None) == inv


@pytest.mark.parametrize("written", [False, True])
def test_binding_refuses_rows_whose_gradient_would_be_lost(written):
    x = torch.zeros(5, 6, 64, dtype=torch.bfloat16, requires_grad=True)
    for t in (x, x * 2, x[:, :3]):
        with pytest.raises(ValueError, match="requires grad"):
            cg._bf16_rows(t, CPU, tuple(t.shape), "q", written)
        cg._bf16_rows(t.detach(), CPU, tuple(t.shape), "q", written)
        with torch.no_grad():
            cg._bf16_rows(t, CPU, tuple(t.shape), "q", written)
        with torch.inference_mode():
            cg._bf16_rows(t, CPU, tuple(t.shape), "q", written)


def test_binding_refuses_numbers_that_their_type_does_not_hold():
    """ctypes would take 2^32 + 1 layers for one, and 2^32 for layer 0."""
    for x in (2 ** 31, -2 ** 31 - 1, 2 ** 32):
        with pytest.raises(ValueError, match="32 bits"):
            cg._int32(x, "layer")
    assert cg._int32(2 ** 31 - 1, "layer") == 2 ** 31 - 1
    for i in range(6):
        sizes = [1, 2, 16, 1, 64, 32]
        sizes[i] += 2 ** 32
        with pytest.raises(ValueError, match="32 bits"):
            cg.Int4Cache(*sizes, device="cpu")
