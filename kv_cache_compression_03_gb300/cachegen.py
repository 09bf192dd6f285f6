"""Python binding of the CacheGen codec's C ABI (include/cachegen.h).

The functions named ``cg_*`` mirror the C entry points one to one and only
marshal arguments: every step of encoding and decoding runs in the CUDA
kernels of ``libcachegen.so``. Device buffers are torch tensors (torch is
used for device memory and streams only). There is no CPU fallback: if the
library is missing or no GPU is present, the calls raise.

``Codec`` wraps a plan with its buffers for the common case; ``preset_specs``
gives the per-layer bin counts of the LMCache presets ("LMCache 中的 KV Cache
压缩：CacheGen 编解码原理、配置方式与源码解析", §1: the first 10 K layers and the
first 2 V layers use 32 bins, the rest 16; fewer than 10 layers: all 32).
"""
from __future__ import annotations

import contextlib
import ctypes as ct
import os
import struct
import threading
from dataclasses import dataclass

CG_OK, CG_ERR_INVALID_ARG, CG_ERR_SPEC, CG_ERR_CAPACITY = 0, 1, 2, 3
CG_ERR_NONFINITE, CG_ERR_CORRUPT, CG_ERR_TIMEOUT, CG_ERR_CUDA, CG_ERR_UNSUPPORTED = 4, 5, 6, 7, 8


class cg_quant_spec(ct.Structure):
    _fields_ = [("start_layer", ct.c_int32), ("end_layer", ct.c_int32), ("bins", ct.c_int32)]


class cg_config(ct.Structure):
    _fields_ = [("num_layers", ct.c_int32), ("num_tokens", ct.c_int32),
                ("num_heads", ct.c_int32), ("head_size", ct.c_int32),
                ("chunk_tokens", ct.c_int32),
                ("kspecs", ct.POINTER(cg_quant_spec)), ("n_kspecs", ct.c_int32),
                ("vspecs", ct.POINTER(cg_quant_spec)), ("n_vspecs", ct.c_int32)]


class cg_sizes(ct.Structure):
    _fields_ = [("workspace_bytes", ct.c_size_t), ("max_stream_bytes", ct.c_size_t),
                ("cdf_entries", ct.c_size_t), ("num_streams", ct.c_size_t),
                ("num_scales", ct.c_size_t), ("raw_bytes", ct.c_size_t),
                ("num_groups", ct.c_int32), ("num_tiles", ct.c_int32),
                ("encode_launches", ct.c_int32), ("decode_launches", ct.c_int32),
                ("num_objects", ct.c_int32)]


class cg_encoded(ct.Structure):
    _fields_ = [("bytestream", ct.c_void_p), ("bytestream_capacity", ct.c_size_t),
                ("lengths", ct.c_void_p), ("cdf", ct.c_void_p), ("amax", ct.c_void_p)]


class cg_kernel_profile(ct.Structure):
    _fields_ = [("kernel", ct.c_char_p), ("launches", ct.c_int64), ("total_ms", ct.c_double)]


class cg_int4_cache(ct.Structure):
    _fields_ = [("data", ct.c_void_p), ("status", ct.c_void_p), ("num_layers", ct.c_int32),
                ("num_pages", ct.c_int32), ("page_tokens", ct.c_int32), ("num_heads", ct.c_int32),
                ("head_size", ct.c_int32), ("group", ct.c_int32)]


class cg_kv_rows(ct.Structure):
    _fields_ = [("k", ct.c_void_p), ("v", ct.c_void_p)] + \
        [(n, ct.c_int64) for n in ("k_layer_stride", "k_token_stride", "k_head_stride",
                                   "v_layer_stride", "v_token_stride", "v_head_stride")]


class cg_page_batch(ct.Structure):
    _fields_ = [("block_table", ct.c_void_p), ("table_stride", ct.c_int64),
                ("table_width", ct.c_int32), ("requests", ct.c_int32),
                ("lens", ct.c_void_p), ("counts", ct.c_void_p), ("free_pages", ct.c_void_p),
                ("free_count", ct.c_void_p), ("free_capacity", ct.c_int32),
                ("num_pages", ct.c_int32), ("page_tokens", ct.c_int32),
                ("cu_out", ct.c_void_p), ("lens_out", ct.c_void_p),
                ("free_count_out", ct.c_void_p), ("slots_out", ct.c_void_p),
                ("tokens", ct.c_int64), ("status", ct.c_void_p)]


class cg_attention(ct.Structure):
    _fields_ = [("q", ct.c_void_p), ("q_token_stride", ct.c_int64), ("q_head_stride", ct.c_int64),
                ("out", ct.c_void_p), ("out_token_stride", ct.c_int64),
                ("out_head_stride", ct.c_int64), ("cu_q", ct.c_void_p), ("kv_lens", ct.c_void_p),
                ("block_table", ct.c_void_p), ("table_stride", ct.c_int64),
                ("table_width", ct.c_int32), ("requests", ct.c_int32), ("tokens", ct.c_int32),
                ("q_heads", ct.c_int32), ("max_q_len", ct.c_int32), ("window", ct.c_int32),
                ("sinks", ct.c_int32), ("scale", ct.c_float)]


class cg_token_weights(ct.Structure):
    _fields_ = [("in_", ct.c_void_p), ("out", ct.c_void_p)] + \
        [(n, ct.c_int64) for n in ("in_request_stride", "in_head_stride", "out_request_stride",
                                   "out_head_stride")] + [("width", ct.c_int32)]


class cg_token_choice(ct.Structure):
    _fields_ = [("weights", ct.c_void_p), ("layer_stride", ct.c_int64),
                ("request_stride", ct.c_int64), ("head_stride", ct.c_int64),
                ("layers", ct.c_int32), ("requests", ct.c_int32), ("heads", ct.c_int32),
                ("width", ct.c_int32), ("lens", ct.c_void_p), ("budget", ct.c_int32),
                ("recent", ct.c_int32), ("sinks", ct.c_int32), ("kept", ct.c_void_p),
                ("lens_out", ct.c_void_p), ("status", ct.c_void_p)]


class cg_compaction(ct.Structure):
    _fields_ = [("kept", ct.c_void_p), ("kept_layer_stride", ct.c_int64),
                ("kept_request_stride", ct.c_int64), ("kept_head_stride", ct.c_int64),
                ("weights", ct.c_void_p), ("weights_layer_stride", ct.c_int64),
                ("weights_request_stride", ct.c_int64), ("weights_head_stride", ct.c_int64),
                ("weights_width", ct.c_int32), ("budget", ct.c_int32), ("layers", ct.c_int32),
                ("requests", ct.c_int32), ("lens", ct.c_void_p), ("new_lens", ct.c_void_p),
                ("block_table", ct.c_void_p), ("table_stride", ct.c_int64),
                ("table_width", ct.c_int32)]


class cg_page_release(ct.Structure):
    _fields_ = [("block_table", ct.c_void_p), ("table_stride", ct.c_int64),
                ("table_width", ct.c_int32), ("requests", ct.c_int32), ("lens", ct.c_void_p),
                ("new_lens", ct.c_void_p), ("free_pages", ct.c_void_p),
                ("free_count", ct.c_void_p), ("free_capacity", ct.c_int32),
                ("num_pages", ct.c_int32), ("page_tokens", ct.c_int32), ("cu_out", ct.c_void_p),
                ("lens_out", ct.c_void_p), ("free_count_out", ct.c_void_p),
                ("status", ct.c_void_p)]


class CacheGenError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {cg_status_string(status)} ({status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libcachegen.so")


def load(build_if_missing: bool = True) -> ct.CDLL:
    """Load libcachegen.so (building it with nvcc when absent)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if build_if_missing:
            from . import build as _build
            path = _build.build()
        _lib = _open(path)
        return _lib


@contextlib.contextmanager
def use_library(path: str):
    """Run the calls of this module against another build of the library
    (the tests' variants with forced slow paths), then switch back."""
    global _lib
    L = _open(path)
    with _lock:
        prev, _lib = _lib, L
    try:
        yield L
    finally:
        with _lock:
            _lib = prev


def _open(path: str) -> ct.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libcachegen.so not found at {path}; run build() first")
    L = ct.CDLL(path)
    P, sz, u64 = ct.c_void_p, ct.c_size_t, ct.c_uint64
    st = ct.c_int
    sigs = {
        "cg_plan_create": (st, [ct.POINTER(cg_config), ct.POINTER(ct.c_void_p)]),
        "cg_plan_destroy": (None, [P]),
        "cg_plan_sizes": (st, [P, ct.POINTER(cg_sizes)]),
        "cg_plan_config": (st, [P, ct.POINTER(cg_config), ct.POINTER(cg_quant_spec),
                                ct.c_int32, ct.POINTER(cg_quant_spec), ct.c_int32]),
        "cg_encode": (st, [P, P, P, sz, ct.POINTER(cg_encoded), P]),
        "cg_decode": (st, [P, ct.POINTER(cg_encoded), u64, P, sz, P, P]),
        "cg_last_device_error": (st, [P, P, ct.POINTER(ct.c_int), ct.POINTER(u64), P]),
        "cg_container_size": (st, [P, u64, ct.POINTER(sz)]),
        "cg_serialize": (st, [P, ct.POINTER(cg_encoded), u64, P, sz, ct.POINTER(sz), P]),
        "cg_container_open": (st, [P, sz, ct.POINTER(ct.c_void_p), ct.POINTER(u64)]),
        "cg_deserialize": (st, [P, P, sz, ct.POINTER(cg_encoded), P]),
        "cg_status_string": (ct.c_char_p, [st]),
        "cg_encode_noalloc": (st, [P, P, ct.POINTER(cg_encoded), P, P]),
        "cg_object_range": (st, [P, ct.c_int32, ct.POINTER(ct.c_int32),
                                 ct.POINTER(ct.c_int32)]),
        "cg_object_streams": (st, [P, P, ct.c_int32, ct.POINTER(u64), ct.POINTER(u64), P]),
        "cg_object_container_size": (st, [P, ct.c_int32, u64, ct.POINTER(sz)]),
        "cg_serialize_object": (st, [P, ct.POINTER(cg_encoded), P, ct.c_int32, P, sz,
                                     ct.POINTER(sz), P]),
        "cg_deserialize_objects": (st, [P, ct.c_int32, ct.POINTER(ct.c_void_p),
                                        ct.POINTER(sz), ct.POINTER(cg_encoded),
                                        ct.POINTER(u64), P]),
        "cg_int8_encode": (st, [P, ct.c_int64, ct.c_int32, P, P, P, P]),
        "cg_int8_decode": (st, [P, P, ct.c_int64, ct.c_int32, P, P]),
        "cg_int4_cache_bytes": (st, [ct.POINTER(cg_int4_cache), ct.POINTER(sz)]),
        "cg_int4_take_error": (st, [ct.POINTER(cg_int4_cache), P, P]),
        # the structs of rows, batches and attention calls come as packed bytes
        "cg_int4_store": (st, [ct.POINTER(cg_int4_cache), ct.c_int32, ct.c_int32, P, P,
                               ct.c_int64, P]),
        "cg_int4_load": (st, [ct.POINTER(cg_int4_cache), ct.c_int32, ct.c_int32, P, P,
                              ct.c_int64, P]),
        "cg_pages_grow": (st, [P, P]),
        "cg_int4_attention_workspace": (st, [ct.POINTER(cg_int4_cache), P, ct.POINTER(sz)]),
        "cg_int4_attention": (st, [ct.POINTER(cg_int4_cache), ct.c_int32, P, P, sz, P]),
        "cg_int4_attention_shared_workspace": (st, [ct.POINTER(cg_int4_cache), P, ct.c_int32,
                                                    ct.POINTER(sz)]),
        "cg_int4_attention_shared": (st, [ct.POINTER(cg_int4_cache), ct.c_int32, P, ct.c_int32, P,
                                          sz, P]),
        "cg_int4_weigh_workspace": (st, [ct.POINTER(cg_int4_cache), P, P, ct.POINTER(sz)]),
        "cg_int4_weigh": (st, [ct.POINTER(cg_int4_cache), ct.c_int32, P, P, P, sz, P]),
        "cg_choose_tokens": (st, [P, P]),
        "cg_int4_compact": (st, [ct.POINTER(cg_int4_cache), ct.c_int32, P, P]),
        "cg_pages_release": (st, [P, P]),
        "cg_profile_enable": (st, [P, ct.c_int32]),
        "cg_profile_read": (st, [P, ct.POINTER(cg_kernel_profile), ct.c_int32,
                                 ct.POINTER(ct.c_int32)]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


def _check(st: int, what: str):
    if st != CG_OK:
        raise CacheGenError(st, what)


def _stream_handle(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ct.c_void_p(s.cuda_stream)


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


def _check_status_buffer(status_out, what: str) -> None:
    """The C side copies a 16-byte status block into status_out: it must be
    a CUDA tensor of at least 16 bytes (a smaller one would be overrun)."""
    if status_out is None or not getattr(status_out, "is_cuda", False):
        raise ValueError(f"{what}: status_out must be a CUDA tensor")
    if status_out.numel() * status_out.element_size() < 16:
        raise ValueError(f"{what}: status_out must hold at least 16 bytes")


# ------------------------------------------------------------ C ABI mirror

def cg_status_string(status: int) -> str:
    try:
        return load(build_if_missing=False).cg_status_string(status).decode()
    except Exception:  # library not loadable: still give a message
        return f"status {status}"


def _specs_array(specs):
    arr = (cg_quant_spec * len(specs))()
    for i, (s, e, b) in enumerate(specs):
        arr[i] = cg_quant_spec(int(s), int(e), int(b))
    return arr


def cg_plan_create(num_layers, num_tokens, num_heads, head_size, chunk_tokens, kspecs, vspecs):
    """Validate a configuration and return an opaque plan handle (int)."""
    ka, va = _specs_array(kspecs), _specs_array(vspecs)
    cfg = cg_config(num_layers, num_tokens, num_heads, head_size, chunk_tokens,
                    ka, len(kspecs), va, len(vspecs))
    h = ct.c_void_p()
    _check(load().cg_plan_create(ct.byref(cfg), ct.byref(h)), "cg_plan_create")
    return h.value


def cg_plan_destroy(plan) -> None:
    if plan:
        load().cg_plan_destroy(ct.c_void_p(plan))


def cg_plan_sizes(plan) -> cg_sizes:
    s = cg_sizes()
    _check(load().cg_plan_sizes(ct.c_void_p(plan), ct.byref(s)), "cg_plan_sizes")
    return s


def cg_plan_config(plan):
    """The configuration of a plan: (num_layers, num_tokens, num_heads,
    head_size, chunk_tokens, kspecs, vspecs) with the specs as
    (start_layer, end_layer, bins) triples."""
    lib = load()
    cfg = cg_config()
    st = lib.cg_plan_config(ct.c_void_p(plan), ct.byref(cfg), None, 0, None, 0)
    if st not in (CG_OK, CG_ERR_CAPACITY):
        _check(st, "cg_plan_config")
    ka = (cg_quant_spec * max(cfg.n_kspecs, 1))()
    va = (cg_quant_spec * max(cfg.n_vspecs, 1))()
    _check(lib.cg_plan_config(ct.c_void_p(plan), ct.byref(cfg), ka, cfg.n_kspecs, va,
                              cfg.n_vspecs), "cg_plan_config")
    ks = [(ka[i].start_layer, ka[i].end_layer, ka[i].bins) for i in range(cfg.n_kspecs)]
    vs = [(va[i].start_layer, va[i].end_layer, va[i].bins) for i in range(cfg.n_vspecs)]
    return (cfg.num_layers, cfg.num_tokens, cfg.num_heads, cfg.head_size, cfg.chunk_tokens,
            ks, vs)


def _encoded_struct(bytestream, lengths, cdf, amax) -> cg_encoded:
    return cg_encoded(_ptr(bytestream), bytestream.numel() * bytestream.element_size(),
                      _ptr(lengths), _ptr(cdf), _ptr(amax))


def cg_encode(plan, kv, workspace, bytestream, lengths, cdf, amax, stream=None) -> None:
    enc = _encoded_struct(bytestream, lengths, cdf, amax)
    _check(load().cg_encode(ct.c_void_p(plan), ct.c_void_p(_ptr(kv)), ct.c_void_p(_ptr(workspace)),
                            workspace.numel(), ct.byref(enc), _stream_handle(stream)), "cg_encode")


def cg_encode_noalloc(plan, kv, bytestream, lengths, cdf, amax, status_out, stream=None) -> None:
    """cg_encode with the library's fixed scratch array instead of a
    workspace, for callers that cannot allocate device memory at encode time
    (see include/cachegen.h). status_out: a device tensor of >= 16 bytes that
    receives the status word and total stream bytes; read it with
    cg_last_device_error(plan, status_out)."""
    _check_status_buffer(status_out, "cg_encode_noalloc")
    enc = _encoded_struct(bytestream, lengths, cdf, amax)
    _check(load().cg_encode_noalloc(ct.c_void_p(plan), ct.c_void_p(_ptr(kv)), ct.byref(enc),
                                    ct.c_void_p(_ptr(status_out)), _stream_handle(stream)),
           "cg_encode_noalloc")


def cg_decode(plan, bytestream, lengths, cdf, amax, stream_bytes, workspace, kv_out,
              stream=None) -> None:
    enc = _encoded_struct(bytestream, lengths, cdf, amax)
    _check(load().cg_decode(ct.c_void_p(plan), ct.byref(enc), int(stream_bytes),
                            ct.c_void_p(_ptr(workspace)), workspace.numel(),
                            ct.c_void_p(_ptr(kv_out)), _stream_handle(stream)), "cg_decode")


def cg_int8_encode(kv, rows, channels, q_out, scales_out, status_out, stream=None) -> None:
    """Int8 baseline encode (include/cachegen.h): kv bf16 [rows][channels]
    into q_out int8 [rows][channels] and scales_out fp32 [rows]; status_out
    (>= 16 bytes) gets the device status, read with
    cg_last_device_error(None, status_out)."""
    _check_status_buffer(status_out, "cg_int8_encode")
    _check(load().cg_int8_encode(ct.c_void_p(_ptr(kv)), int(rows), int(channels),
                                 ct.c_void_p(_ptr(q_out)), ct.c_void_p(_ptr(scales_out)),
                                 ct.c_void_p(_ptr(status_out)), _stream_handle(stream)),
           "cg_int8_encode")


def cg_int8_decode(q, scales, rows, channels, kv_out, stream=None) -> None:
    """Int8 baseline decode: q int8 [rows][channels] and scales fp32 [rows]
    into kv_out bf16 [rows][channels]."""
    _check(load().cg_int8_decode(ct.c_void_p(_ptr(q)), ct.c_void_p(_ptr(scales)), int(rows),
                                 int(channels), ct.c_void_p(_ptr(kv_out)), _stream_handle(stream)),
           "cg_int8_decode")


def cg_object_range(plan, obj):
    """(first token, token count) of an object of the plan."""
    t0, n = ct.c_int32(0), ct.c_int32(0)
    _check(load().cg_object_range(ct.c_void_p(plan), int(obj), ct.byref(t0), ct.byref(n)),
           "cg_object_range")
    return t0.value, n.value


def cg_object_streams(plan, workspace, obj, stream=None):
    """(offset, bytes) of an object's streams in the last encoded bytestream."""
    off, nb = ct.c_uint64(0), ct.c_uint64(0)
    _check(load().cg_object_streams(ct.c_void_p(plan), ct.c_void_p(_ptr(workspace)), int(obj),
                                    ct.byref(off), ct.byref(nb), _stream_handle(stream)),
           "cg_object_streams")
    return off.value, nb.value


def cg_object_container_size(plan, obj, stream_bytes) -> int:
    n = ct.c_size_t(0)
    _check(load().cg_object_container_size(ct.c_void_p(plan), int(obj), int(stream_bytes),
                                           ct.byref(n)), "cg_object_container_size")
    return n.value


def cg_serialize_object(plan, bytestream, lengths, cdf, amax, workspace, obj, host_out,
                        stream=None) -> int:
    enc = _encoded_struct(bytestream, lengths, cdf, amax)
    w = ct.c_size_t(0)
    _check(load().cg_serialize_object(ct.c_void_p(plan), ct.byref(enc),
                                      ct.c_void_p(_ptr(workspace)), int(obj),
                                      ct.c_void_p(host_out.data_ptr()), host_out.numel(),
                                      ct.byref(w), _stream_handle(stream)), "cg_serialize_object")
    return w.value


def cg_deserialize_objects(plan, hosts, bytestream, lengths, cdf, amax, stream=None) -> int:
    """hosts: uint8 CPU tensors, one container per object in object order.
    Returns the total stream bytes."""
    n = len(hosts)
    ptrs = (ct.c_void_p * max(n, 1))(*[h.data_ptr() for h in hosts])
    lens = (ct.c_size_t * max(n, 1))(*[h.numel() for h in hosts])
    enc = _encoded_struct(bytestream, lengths, cdf, amax)
    sb = ct.c_uint64(0)
    _check(load().cg_deserialize_objects(ct.c_void_p(plan), n, ptrs, lens, ct.byref(enc),
                                         ct.byref(sb), _stream_handle(stream)),
           "cg_deserialize_objects")
    return sb.value


def int8_encode(kv, stream=None, sync: bool = True):
    """Int8 baseline encode of a contiguous bf16 cuda tensor whose last
    dimension is the row (a KV cache [L, 2, T, H, D] is taken as rows of
    H*D). Returns (q int8 of kv's shape, scales fp32 [rows], status tensor);
    with sync, a device error is raised."""
    import torch
    assert kv.dtype == torch.bfloat16 and kv.is_cuda and kv.is_contiguous()
    C = kv.shape[-1] if kv.dim() != 5 else kv.shape[-2] * kv.shape[-1]
    rows = kv.numel() // C if C else 0
    q = torch.empty(kv.shape, dtype=torch.int8, device=kv.device)
    scales = torch.empty(rows, dtype=torch.float32, device=kv.device)
    status = torch.empty(16, dtype=torch.uint8, device=kv.device)
    cg_int8_encode(kv, rows, C, q, scales, status, stream)
    if sync:
        st, _ = cg_last_device_error(None, status, stream)
        _check(st, "cg_int8_encode (device)")
    return q, scales, status


def int8_decode(q, scales, stream=None):
    """Int8 baseline decode: the bf16 tensor of q's shape."""
    import torch
    C = q.shape[-1] if q.dim() != 5 else q.shape[-2] * q.shape[-1]
    rows = q.numel() // C if C else 0
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    cg_int8_decode(q, scales, rows, C, out, stream)
    return out


def cg_last_device_error(plan, workspace, stream=None):
    """Wait for the stream; return (device status, total stream bytes)."""
    st = ct.c_int(0)
    tot = ct.c_uint64(0)
    _check(load().cg_last_device_error(ct.c_void_p(plan or 0), ct.c_void_p(_ptr(workspace)),
                                       ct.byref(st), ct.byref(tot), _stream_handle(stream)),
           "cg_last_device_error")
    return st.value, tot.value


def cg_container_size(plan, stream_bytes) -> int:
    n = ct.c_size_t(0)
    _check(load().cg_container_size(ct.c_void_p(plan), int(stream_bytes), ct.byref(n)),
           "cg_container_size")
    return n.value


def cg_serialize(plan, bytestream, lengths, cdf, amax, stream_bytes, host_out, stream=None) -> int:
    """Write the container into host_out (a uint8 CPU tensor, ideally
    pinned); returns the bytes written."""
    enc = _encoded_struct(bytestream, lengths, cdf, amax)
    n = ct.c_size_t(0)
    _check(load().cg_serialize(ct.c_void_p(plan), ct.byref(enc), int(stream_bytes),
                               ct.c_void_p(host_out.data_ptr()), host_out.numel(), ct.byref(n),
                               _stream_handle(stream)), "cg_serialize")
    return n.value


def cg_container_open(host_in):
    """Parse a container header (uint8 CPU tensor); return (plan, stream_bytes)."""
    h = ct.c_void_p()
    sb = ct.c_uint64(0)
    _check(load().cg_container_open(ct.c_void_p(host_in.data_ptr()), host_in.numel(),
                                    ct.byref(h), ct.byref(sb)), "cg_container_open")
    return h.value, sb.value


def cg_deserialize(plan, host_in, bytestream, lengths, cdf, amax, stream=None) -> None:
    enc = _encoded_struct(bytestream, lengths, cdf, amax)
    _check(load().cg_deserialize(ct.c_void_p(plan), ct.c_void_p(host_in.data_ptr()),
                                 host_in.numel(), ct.byref(enc), _stream_handle(stream)),
           "cg_deserialize")


def cg_profile_enable(plan, max_launches: int) -> None:
    _check(load().cg_profile_enable(ct.c_void_p(plan), int(max_launches)), "cg_profile_enable")


def cg_profile_read(plan) -> dict:
    """{kernel name: (launches, total ms)} since the last read."""
    arr = (cg_kernel_profile * 16)()
    n = ct.c_int32(0)
    _check(load().cg_profile_read(ct.c_void_p(plan), arr, 16, ct.byref(n)), "cg_profile_read")
    return {arr[i].kernel.decode(): (int(arr[i].launches), float(arr[i].total_ms))
            for i in range(min(n.value, 16))}


# ------------------------------------------------------------- convenience

def preset_specs(num_layers: int):
    """(kspecs, vspecs) of the LMCache presets for a model with num_layers
    layers: K's first 10 and V's first 2 layers at 32 bins, the rest at 16;
    with fewer than 10 layers every layer uses 32 bins."""
    L = int(num_layers)
    if L <= 0:
        raise ValueError("num_layers must be positive")
    if L < 10:
        return [(0, L, 32)], [(0, L, 32)]
    k = [(0, 10, 32)] + ([(10, L, 16)] if L > 10 else [])
    v = [(0, 2, 32), (2, L, 16)]
    return k, v


@dataclass
class Encoded:
    """Device buffers of one encoded KV blob."""
    bytestream: "object"   # uint8 [capacity]
    lengths: "object"      # int32 [2*L*T]
    cdf: "object"          # uint16 (stored as int16) [cdf_entries]
    amax: "object"         # float32 [2, L, T]
    stream_bytes: int

    def nbytes(self) -> int:
        return int(self.stream_bytes) + self.lengths.numel() * 4 + self.cdf.numel() * 2 + \
            self.amax.numel() * 4


class Codec:
    """A plan plus its device buffers, for encoding/decoding one shape."""

    def __init__(self, num_layers, num_tokens, num_heads, head_size, chunk_tokens=256,
                 kspecs=None, vspecs=None, device="cuda"):
        import torch
        if kspecs is None or vspecs is None:
            k, v = preset_specs(num_layers)
            kspecs = kspecs or k
            vspecs = vspecs or v
        self.L, self.T, self.H, self.D = num_layers, num_tokens, num_heads, head_size
        self.chunk_tokens = chunk_tokens
        self.kspecs, self.vspecs = list(kspecs), list(vspecs)
        self.plan = cg_plan_create(num_layers, num_tokens, num_heads, head_size, chunk_tokens,
                                   self.kspecs, self.vspecs)
        self.sizes = cg_plan_sizes(self.plan)
        self.device = torch.device(device)
        self.workspace = torch.empty(self.sizes.workspace_bytes, dtype=torch.uint8,
                                     device=self.device)

    def __del__(self):
        try:
            cg_plan_destroy(self.plan)
        except Exception:
            pass

    def alloc_encoded(self, capacity=None) -> Encoded:
        import torch
        cap = int(capacity or self.sizes.max_stream_bytes)
        cap = (cap + 15) // 16 * 16
        d = self.device
        return Encoded(torch.empty(cap, dtype=torch.uint8, device=d),
                       torch.empty(self.sizes.num_streams, dtype=torch.int32, device=d),
                       torch.empty(self.sizes.cdf_entries, dtype=torch.int16, device=d),
                       torch.empty((2, self.L, self.T), dtype=torch.float32, device=d), 0)

    def encode(self, kv, out: Encoded | None = None, sync: bool = True, stream=None) -> Encoded:
        """kv: bf16 cuda tensor [L, 2, T, H, D] (contiguous)."""
        import torch
        assert kv.dtype == torch.bfloat16 and kv.is_cuda and kv.is_contiguous()
        assert kv.numel() == self.sizes.raw_bytes // 2
        out = out or self.alloc_encoded()
        cg_encode(self.plan, kv, self.workspace, out.bytestream, out.lengths, out.cdf, out.amax,
                  stream)
        if sync:
            st, total = cg_last_device_error(self.plan, self.workspace, stream)
            _check(st, "cg_encode (device)")
            out.stream_bytes = total
        return out

    def decode(self, enc: Encoded, kv_out=None, sync: bool = True, stream=None):
        import torch
        if kv_out is None:
            kv_out = torch.empty((self.L, 2, self.T, self.H, self.D), dtype=torch.bfloat16,
                                 device=self.device)
        cg_decode(self.plan, enc.bytestream, enc.lengths, enc.cdf, enc.amax, enc.stream_bytes,
                  self.workspace, kv_out, stream)
        if sync:
            st, _ = cg_last_device_error(self.plan, self.workspace, stream)
            _check(st, "cg_decode (device)")
        return kv_out

    def to_bytes(self, enc: Encoded, host_out=None, stream=None):
        """Serialise to a uint8 CPU tensor (pinned unless host_out is given)."""
        import torch
        n = cg_container_size(self.plan, enc.stream_bytes)
        if host_out is None:
            host_out = torch.empty(n, dtype=torch.uint8, pin_memory=True)
        w = cg_serialize(self.plan, enc.bytestream, enc.lengths, enc.cdf, enc.amax,
                         enc.stream_bytes, host_out, stream)
        return host_out[:w]

    def object_bytes(self, enc: Encoded, stream=None):
        """One container per object (uint8 CPU tensors) of the blob that the
        last encode with this codec wrote into enc."""
        import torch
        out = []
        for o in range(self.sizes.num_objects):
            _, nb = cg_object_streams(self.plan, self.workspace, o, stream)
            host = torch.empty(cg_object_container_size(self.plan, o, nb), dtype=torch.uint8,
                               pin_memory=True)
            w = cg_serialize_object(self.plan, enc.bytestream, enc.lengths, enc.cdf, enc.amax,
                                    self.workspace, o, host, stream)
            out.append(host[:w])
        return out

    def from_object_bytes(self, hosts, out: Encoded | None = None, stream=None) -> Encoded:
        """Put the containers of all objects back for one decode."""
        out = out or self.alloc_encoded()
        out.stream_bytes = cg_deserialize_objects(self.plan, hosts, out.bytestream, out.lengths,
                                                  out.cdf, out.amax, stream)
        return out

    @staticmethod
    def from_bytes(host_in, device="cuda", stream=None):
        """Open a container (uint8 CPU tensor); return (codec, encoded)."""
        plan, sb = cg_container_open(host_in)
        try:
            L, T, H, D, ch, kspecs, vspecs = cg_plan_config(plan)
        finally:
            cg_plan_destroy(plan)
        codec = Codec(L, T, H, D, ch, kspecs, vspecs, device=device)
        enc = codec.alloc_encoded(capacity=max(16, sb))
        enc.stream_bytes = sb
        cg_deserialize(codec.plan, host_in, enc.bytestream, enc.lengths, enc.cdf, enc.amax,
                       stream)
        return codec, enc


# ---------------------------------------------- paged cache held in 4 bits
# These calls run once per layer and decode step, where a microsecond of Python
# is a microsecond of the step: checks are written out on plain tuples, and the
# structs of the C calls are packed in one go (their layout is asserted here).

_torch = None   # the module, once one of these calls needs it
_ROWS = struct.Struct("@PPqqqqqq")
_BATCH = struct.Struct("@PqiiPPPPiiiPPPPqP")
_ATTENTION = struct.Struct("@PqqPqqPPPqiiiiiiif")
_WEIGHTS = struct.Struct("@PPqqqqi")
_CHOICE = struct.Struct("@PqqqiiiiPiiiPPP")
_COMPACTION = struct.Struct("@PqqqPqqqiiiiPPPqi")
_RELEASE = struct.Struct("@PqiiPPPPiiiPPPP")
assert all(-(-s.size // 8) * 8 == ct.sizeof(t) for s, t in (
    (_ROWS, cg_kv_rows), (_BATCH, cg_page_batch), (_ATTENTION, cg_attention),
    (_WEIGHTS, cg_token_weights), (_CHOICE, cg_token_choice), (_COMPACTION, cg_compaction),
    (_RELEASE, cg_page_release)))


def _need_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _on_stream(stream, fn, *args, **kw):
    """fn(*args, **kw) with `stream` current: its temporaries and outputs are
    then that stream's too. The tensors passed in (and the cache's own) may be
    another stream's: their memory is not handed out again before the call on
    this one has ended, however soon the caller drops them."""
    torch = _torch or _need_torch()
    with torch.cuda.stream(stream):
        res = fn(*args, **kw)
    owner = getattr(fn, "__self__", None)
    used = [owner.data, owner.status] if owner is not None else []
    for a in args:
        used += vars(a).values() if isinstance(a, (PagePlan, KeptTokens, ReleasePlan)) else [a]
    for t in used:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return res


class _Launch:
    """The current stream of a device (its index), with that device made
    current while a call is enqueued."""
    __slots__ = ("index", "back")

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        C = _torch._C
        now = C._cuda_getDevice()
        if now != self.index:
            _torch.cuda.set_device(self.index)
            self.back = now
        else:
            self.back = -1
        return C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.back >= 0:
            _torch.cuda.set_device(self.back)


def _need(cond, what: str):
    if not cond:
        raise ValueError(what)


def _int32(x, what: str) -> int:
    """x, an int that a 32-bit argument holds (ctypes would cut a larger one off)."""
    if not -0x80000000 <= x <= 0x7FFFFFFF:
        raise ValueError(f"{what} must fit 32 bits")
    return x


def _ints(t, device, shape, what: str) -> int:
    """The address of a contiguous int32 tensor of the given shape on the device."""
    torch = _torch or _need_torch()
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.shape == shape and
            t.device == device and t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {list(shape)} on {device}")
    return t.data_ptr()


def _table(t, device, what: str):
    """(requests, entries of a row, elements between rows) of a block table."""
    torch = _torch or _need_torch()
    if isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == device and t.dim() == 2:
        n, width = t.shape
        s0, s1 = t.stride()
        if n == 0 or ((s1 == 1 or width <= 1) and (s0 >= width or n <= 1)):
            return n, width, s0 if n > 1 else width
    raise ValueError(f"{what} must be an int32 tensor [requests, pages] on {device}, a row's "
                     f"entries adjacent")


def _bf16_rows(t, device, shape, what: str, written: bool):
    """(address, strides but the last) of a bf16 tensor [.., head_size] of the
    given shape whose rows the kernels can read (and, when written, that do
    not overlap). A dimension of one element counts stride 0. No gradient flows
    through the cache: a tensor that autograd would follow is refused."""
    torch = _torch or _need_torch()
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.shape == shape and
            t.device == device):
        raise ValueError(f"{what} must be a bf16 tensor of shape {list(shape)} on {device}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires grad, and no gradient flows through the cache: pass "
                         f"{what}.detach(), or call under torch.no_grad()")
    ptr, strides = t.data_ptr(), t.stride()
    last = strides[-1]
    strides = [s if n > 1 else 0 for s, n in zip(strides[:-1], shape)]
    if t.numel() == 0:
        return ptr, strides
    bits = ptr >> 1
    for s in strides:
        bits |= s
    if last != 1 or bits & 7:
        raise ValueError(f"{what}: channels must be adjacent, rows 16-byte aligned")
    if written:
        # each dimension steps over everything inside the smaller ones
        inner = shape[-1]
        for s, n in sorted((s, n) for s, n in zip(strides, shape) if n > 1):
            _need(s >= inner, f"{what}: rows overlap")
            inner += s * (n - 1)
    return ptr, strides


def _floats(t, device, shape, what: str, written: bool):
    """(address, strides but the last) of an fp32 tensor [.., n] of the given
    shape with adjacent elements (and, when written, rows that do not overlap). A dimension of
    one element counts stride 0. Sums of attention weights carry no gradient: a tensor that
    autograd would follow is refused."""
    torch = _torch or _need_torch()
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.shape == shape and
            t.device == device):
        raise ValueError(f"{what} must be an fp32 tensor of shape {list(shape)} on {device}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires grad, and no gradient flows through it: pass {what}.detach(), "
                         f"or call under torch.no_grad()")
    strides = t.stride()
    if shape[-1] > 1 and strides[-1] != 1 and t.numel():
        raise ValueError(f"{what}: elements of a row must be adjacent")
    strides = [s if n > 1 else 0 for s, n in zip(strides[:-1], shape)]
    if written and t.numel():
        inner = shape[-1]
        for s, n in sorted((s, n) for s, n in zip(strides, shape) if n > 1):
            _need(s >= inner, f"{what}: rows overlap")
            inner += s * (n - 1)
    return t.data_ptr(), strides


@dataclass
class PagePlan:
    """What grow_pages found: tensors on the device."""
    slots: "object"        # int32 [tokens], -1 behind the last request
    cu: "object"           # int32 [requests + 1]
    lens: "object"         # int32 [requests], with the new tokens
    free_count: "object"   # int32 [1]
    status: "object"       # uint8 [16]

    def check(self):
        """Wait for the current stream; raise if the pages could not be had."""
        import torch
        with torch.cuda.device(self.status.device):
            st, _ = cg_last_device_error(None, self.status)
        _check(st, "cg_pages_grow (device)")


def grow_pages(block_table, lens, counts, free_pages, free_count, page_tokens: int, tokens: int,
               num_pages: int | None = None, out: PagePlan | None = None, stream=None) -> PagePlan:
    """Pages and slots of a batch's new tokens (cg_pages_grow in
    include/cachegen.h). block_table int32 [requests, width] gets the ids of
    the pages taken; lens and counts are int32 [requests] (tokens held, tokens
    new); free_pages int32 [capacity] holds free_count (int32 [1]) free page
    ids, taken from its end. ``tokens`` is the length of the slot map (at
    least the sum of counts; the rest of it is -1). With ``num_pages`` page
    ids are checked against the cache's size. ``out`` reuses the buffers of an
    earlier plan; its lens and free_count may be the lens and free_count passed
    in (a captured decode loop then advances in place). Enqueues and returns:
    the caller's own check is PagePlan.check(). With ``stream`` the call runs
    there; what made its inputs on another stream must be ordered before it by
    the caller (stream.wait_stream)."""
    if stream is not None:
        return _on_stream(stream, grow_pages, block_table, lens, counts, free_pages, free_count,
                          page_tokens, tokens, num_pages, out)
    torch = _torch or _need_torch()
    _need(isinstance(lens, torch.Tensor) and lens.is_cuda, "lens must be a CUDA tensor")
    dev = lens.device
    n = lens.shape[0] if lens.dim() == 1 else -1
    lens_at, counts_at = _ints(lens, dev, (n,), "lens"), _ints(counts, dev, (n,), "counts")
    rows, width, stride = _table(block_table, dev, "block_table")
    _need(rows == n, "block_table must have one row per request")
    capacity = free_pages.numel()
    free_at = _ints(free_pages, dev, (capacity,), "free_pages")
    nfree_at = _ints(free_count, dev, (1,), "free_count")
    tokens = int(tokens)
    _need(tokens >= 0 and page_tokens > 0, "tokens must not be negative, page_tokens positive")
    if out is None:
        e, i32 = torch.empty, torch.int32
        out = PagePlan(e(tokens, dtype=i32, device=dev), e(n + 1, dtype=i32, device=dev),
                       e(n, dtype=i32, device=dev), e(1, dtype=i32, device=dev),
                       e(16, dtype=torch.uint8, device=dev))
    else:
        _ints(out.slots, dev, (tokens,), "out.slots")
        _ints(out.cu, dev, (n + 1,), "out.cu")
        _ints(out.lens, dev, (n,), "out.lens")
        _ints(out.free_count, dev, (1,), "out.free_count")
        _check_status_buffer(out.status, "grow_pages")
        _need(out.status.device == dev, "out.status must be on the same device")
    try:
        b = _BATCH.pack(block_table.data_ptr(), stride, width, n, lens_at, counts_at, free_at,
                        nfree_at, capacity, 0x7FFFFFFF // page_tokens if num_pages is None else num_pages,
                        page_tokens, out.cu.data_ptr(), out.lens.data_ptr(), out.free_count.data_ptr(),
                        out.slots.data_ptr(), tokens, out.status.data_ptr())
    except struct.error as e:
        raise ValueError(f"a number does not fit its type: {e}") from None
    with _Launch(dev.index) as s:
        st = (_lib or load()).cg_pages_grow(b, s)
    _check(st, "cg_pages_grow")
    return out


@dataclass
class ReleasePlan:
    """What release_pages did: tensors on the device."""
    cu: "object"           # int32 [requests + 1], exclusive sums of the pages released
    lens: "object"         # int32 [requests], the new ones
    free_count: "object"   # int32 [1]
    status: "object"       # 16 bytes

    def check(self):
        """Wait for the current stream; raise if nothing was released."""
        import torch
        with torch.cuda.device(self.status.device):
            st, _ = cg_last_device_error(None, self.status)
        _check(st, "cg_pages_release (device)")


def release_pages(block_table, lens, new_lens, free_pages, free_count, page_tokens: int,
                  num_pages: int | None = None, out: ReleasePlan | None = None,
                  stream=None) -> ReleasePlan:
    """The pages behind shorter requests back to the list of free pages
    (cg_pages_release in include/cachegen.h), the counterpart of grow_pages:
    request r holds lens[r] tokens and keeps new_lens[r] (0 where it ends). free_pages
    (int32 [capacity], free_count of them in use) gets the ids at its end,
    block_table -1 in their place. A page that several requests share may be
    released by one of them only: give the others' new_lens the shared tokens. ``num_pages``
    and ``stream`` as for grow_pages; ``out`` reuses the buffers of an earlier plan, whose
    lens may be lens or new_lens and whose free_count may be free_count."""
    if stream is not None:
        return _on_stream(stream, release_pages, block_table, lens, new_lens, free_pages,
                          free_count, page_tokens, num_pages, out)
    torch = _torch or _need_torch()
    _need(isinstance(lens, torch.Tensor) and lens.is_cuda, "lens must be a CUDA tensor")
    dev = lens.device
    n = lens.shape[0] if lens.dim() == 1 else -1
    lens_at, new_at = _ints(lens, dev, (n,), "lens"), _ints(new_lens, dev, (n,), "new_lens")
    rows, width, stride = _table(block_table, dev, "block_table")
    _need(rows == n, "block_table must have one row per request")
    capacity = free_pages.numel()
    free_at = _ints(free_pages, dev, (capacity,), "free_pages")
    nfree_at = _ints(free_count, dev, (1,), "free_count")
    _need(page_tokens > 0, "page_tokens must be positive")
    if out is None:
        e, i32 = torch.empty, torch.int32
        out = ReleasePlan(e(n + 1, dtype=i32, device=dev), e(n, dtype=i32, device=dev),
                          e(1, dtype=i32, device=dev), e(4, dtype=i32, device=dev))
    else:
        _ints(out.cu, dev, (n + 1,), "out.cu")
        _ints(out.lens, dev, (n,), "out.lens")
        _ints(out.free_count, dev, (1,), "out.free_count")
        _check_status_buffer(out.status, "release_pages")
        _need(out.status.device == dev, "out.status must be on the same device")
    try:
        b = _RELEASE.pack(block_table.data_ptr(), stride, width, n, lens_at, new_at, free_at, nfree_at,
                          capacity, 0x7FFFFFFF // page_tokens if num_pages is None else num_pages,
                          page_tokens, out.cu.data_ptr(), out.lens.data_ptr(),
                          out.free_count.data_ptr(), out.status.data_ptr())
    except struct.error as e:
        raise ValueError(f"a number does not fit its type: {e}") from None
    with _Launch(dev.index) as s:
        st = (_lib or load()).cg_pages_release(b, s)
    _check(st, "cg_pages_release")
    return out


@dataclass
class KeptTokens:
    """What choose_tokens found: tensors on the device."""
    kept: "object"     # int32 [.., requests, heads, budget], ascending, -1 behind the last
    lens: "object"     # int32 [requests]: tokens that stay
    status: "object"   # 16 bytes

    def check(self):
        """Wait for the current stream; raise if a length was wrong."""
        import torch
        with torch.cuda.device(self.status.device):
            st, _ = cg_last_device_error(None, self.status)
        _check(st, "cg_choose_tokens (device)")


def choose_tokens(weights, lens, budget: int, recent: int = 0, sinks: int = 0,
                  out: KeptTokens | None = None, stream=None) -> KeptTokens:
    """The tokens of each head that stay when requests are cut to ``budget``
    tokens (cg_choose_tokens in include/cachegen.h): the first ``sinks``, the last
    ``recent`` and those with the greatest weights (fp32 [requests, heads, n], or
    [layers, requests, heads, n], as Int4Cache.weigh sums them; lens int32 [requests]).
    Of equal weights the lower token stays. ``out`` reuses the buffers of an
    earlier choice; its lens may be lens (Int4Cache.compact wants both). With ``stream`` the call
    runs there."""
    if stream is not None:
        return _on_stream(stream, choose_tokens, weights, lens, budget, recent, sinks, out)
    torch = _torch or _need_torch()
    _need(isinstance(weights, torch.Tensor) and weights.is_cuda and weights.dim() in (3, 4),
          "weights must be a CUDA tensor [requests, heads, tokens], with or without layers")
    dev, shape = weights.device, tuple(weights.shape)
    at, strides = _floats(weights, dev, shape, "weights", False)
    layers = shape[0] if len(shape) == 4 else 1
    if len(shape) == 3:
        strides = [0] + strides
    n, heads, width = shape[-3:]
    lens_at = _ints(lens, dev, (n,), "lens")
    _need(0 <= _int32(budget, "budget"), "budget must not be negative")
    if out is None:
        e, i32 = torch.empty, torch.int32
        out = KeptTokens(e(shape[:-1] + (budget,), dtype=i32, device=dev), e(n, dtype=i32, device=dev),
                         e(4, dtype=i32, device=dev))
    else:
        _ints(out.kept, dev, shape[:-1] + (budget,), "out.kept")
        _ints(out.lens, dev, (n,), "out.lens")
        _check_status_buffer(out.status, "choose_tokens")
        _need(out.status.device == dev, "out.status must be on the same device")
    try:
        c = _CHOICE.pack(at, *strides, layers, n, heads, width, lens_at, budget, recent, sinks,
                         out.kept.data_ptr(), out.lens.data_ptr(), out.status.data_ptr())
    except struct.error as e:
        raise ValueError(f"a number does not fit its type: {e}") from None
    with _Launch(dev.index) as s:
        st = (_lib or load()).cg_choose_tokens(c, s)
    _check(st, "cg_choose_tokens")
    return out


class Int4Cache:
    """A paged KV cache held in 4 bits, and the attention that reads it
    (cg_int4_* in include/cachegen.h, which defines the format). ``data`` is
    the cache's bytes, uint8 of any shape (made, and zeroed, if not given).

    For serving: no gradient flows through the cache, and rows that require one
    are refused. Calls enqueue on the current stream (or on stream=) and return; errors
    that the GPU finds are kept until check() raises them. Calls that touch
    the same slots, one of them a store, must be ordered by the caller, and so
    must a call with stream= and what made its inputs on another stream
    (stream.wait_stream); the inputs may be dropped once the call has returned."""

    def __init__(self, num_layers, num_pages, page_tokens, num_heads, head_size, group=32,
                 data=None, device="cuda"):
        torch = _torch or _need_torch()
        for x in (num_layers, num_pages, page_tokens, num_heads, head_size, group):
            _int32(x, "a cache's sizes")
        self._c = cg_int4_cache(0, 0, num_layers, num_pages, page_tokens, num_heads, head_size,
                                group)
        self._ref = ct.byref(self._c)
        n = ct.c_size_t(0)
        _check(load().cg_int4_cache_bytes(self._ref, ct.byref(n)), "cg_int4_cache_bytes")
        self.nbytes = n.value
        if data is None:
            data = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)
        _need(isinstance(data, torch.Tensor) and data.is_cuda and data.dtype == torch.uint8 and
              data.is_contiguous() and data.numel() == self.nbytes,
              f"data must be a contiguous uint8 CUDA tensor of {self.nbytes} bytes")
        self.data, self.device = data, data.device
        self.status = torch.zeros(16, dtype=torch.uint8, device=self.device)
        self._c.data, self._c.status = data.data_ptr(), self.status.data_ptr()
        self.num_layers, self.num_pages, self.page_tokens = num_layers, num_pages, page_tokens
        self.num_heads, self.head_size, self.group = num_heads, head_size, group
        self._sizes = {}   # workspaces of attention and weigh, by the sizes that they go by

    def _rows(self, k, v, tokens, layers, written):
        shape = (tokens, self.num_heads, self.head_size)
        if layers is not None:
            shape = (layers,) + shape
        k_at, ks = _bf16_rows(k, self.device, shape, "k", written)
        v_at, vs = _bf16_rows(v, self.device, shape, "v", written)
        if layers is None:
            return _ROWS.pack(k_at, v_at, 0, *ks, 0, *vs)
        return _ROWS.pack(k_at, v_at, *ks, *vs)

    def store(self, k, v, slots, layer: int = 0, stream=None) -> None:
        """Quantise rows k, v (bf16 [tokens, heads, head_size] into one layer,
        or [layers, tokens, heads, head_size] into layers from ``layer`` on;
        kv[:, 0] and kv[:, 1] of Codec.decode's output fit) into the slots
        (int32 [tokens]; -1 skips a token, no other slot may occur twice)."""
        if stream is not None:
            return _on_stream(stream, self.store, k, v, slots, layer)
        shape = k.shape
        _need(len(shape) in (3, 4), "k must be [tokens, heads, head_size], with or without layers")
        tokens, layers = shape[-3], shape[0] if len(shape) == 4 else None
        _int32(layer, "layer")
        rows = self._rows(k, v, tokens, layers, False)
        at = _ints(slots, self.device, (tokens,), "slots")
        with _Launch(self.device.index) as s:
            st = (_lib or load()).cg_int4_store(self._ref, layer, 1 if layers is None else layers,
                                                rows, at, tokens, s)
        _check(st, "cg_int4_store")

    def load(self, slots, layer: int = 0, layers: int | None = None, k_out=None, v_out=None,
             stream=None):
        """The bf16 rows of the slots: (k, v) as [tokens, heads, head_size] of
        one layer, or [layers, tokens, heads, head_size]. Slot -1 gives zeros.
        k_out, v_out take the rows in place (halves of a KV blob for
        Codec.encode, say)."""
        if stream is not None:
            return _on_stream(stream, self.load, slots, layer, layers, k_out, v_out)
        torch = _torch
        tokens = slots.shape[0] if slots.dim() == 1 else -1
        at = _ints(slots, self.device, (tokens,), "slots")
        _int32(layer, "layer")
        H, D = self.num_heads, self.head_size
        shape = (tokens, H, D)
        if layers is not None:
            _need(_int32(layers, "layers") >= 0, "layers must not be negative")
            shape = (layers,) + shape
        if k_out is None and v_out is None:   # what is made here needs no check
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            v_out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            strides = (tokens * H * D, H * D, D)
            rows = _ROWS.pack(k_out.data_ptr(), v_out.data_ptr(), *strides, *strides)
        else:
            if k_out is None:
                k_out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            if v_out is None:
                v_out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
            rows = self._rows(k_out, v_out, tokens, layers, True)
        with _Launch(self.device.index) as s:
            st = (_lib or load()).cg_int4_load(self._ref, layer, 1 if layers is None else layers,
                                               rows, at, tokens, s)
        _check(st, "cg_int4_load")
        return k_out, v_out

    def attention(self, q, cu_q, kv_lens, block_table, layer: int = 0, window: int = 0,
                  sinks: int = 0, scale: float | None = None, max_q_len: int | None = None,
                  out=None, stream=None, shared: int = 0):
        """Attention of the new tokens' queries q (bf16 [tokens, q_heads,
        head_size]) over a layer of the cache: request r owns the rows
        cu_q[r]:cu_q[r + 1] and sees its first kv_lens[r] tokens through row r of
        block_table, causally; with ``window`` only the last ``window`` of
        them and the first ``sinks``. scale defaults to head_size ** -0.5.
        max_q_len, the most rows that any request has, should be given where it is
        small (1 in a decode step): without it kernels for more rows are launched
        too, and a batch of single tokens takes up to 1.7 times as long. Returns
        out, like q; rows from cu_q[-1] on are not written.

        With ``shared``, a multiple of page_tokens, the first ``shared`` tokens of every
        request lie in the same pages (kv_lens counts them, every row of block_table names
        them; those of its first row are read): where there are enough of them they are read
        once for the whole batch. Not with a window. Requests with few rows may then have the
        roundings and the limit on V of those with many (the header names them)."""
        if stream is not None:
            return _on_stream(stream, self.attention, q, cu_q, kv_lens, block_table, layer, window,
                              sinks, scale, max_q_len, out, None, shared)
        torch, dev, D = _torch, self.device, self.head_size
        shape = q.shape
        _need(len(shape) == 3, "q must be [tokens, q_heads, head_size]")
        _int32(layer, "layer")
        tokens, q_heads, _ = shape
        if q_heads <= 0 or q_heads % self.num_heads:
            raise ValueError(f"q_heads must be a multiple of {self.num_heads}")
        shape = (tokens, q_heads, D)
        q_at, (qs0, qs1) = _bf16_rows(q, dev, shape, "q", False)
        n, width, stride = _table(block_table, dev, "block_table")
        lens_at = _ints(kv_lens, dev, (n,), "kv_lens (one entry per row of block_table)")
        cu_at = _ints(cu_q, dev, (n + 1,), "cu_q")
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
            out_at, os0, os1 = out.data_ptr(), q_heads * D, D
        else:
            out_at, (os0, os1) = _bf16_rows(out, dev, shape, "out", True)
        try:
            a = _ATTENTION.pack(q_at, qs0, qs1, out_at, os0, os1, cu_at, lens_at,
                                block_table.data_ptr(), stride, width, n, tokens, q_heads,
                                max_q_len or 0, window, sinks, D ** -0.5 if scale is None else scale)
        except struct.error as e:
            raise ValueError(f"a number does not fit its type: {e}") from None
        L = _lib or load()
        # the size depends on the most rows that a request can have per KV head, and on the cache
        rows = (min(max_q_len, tokens) if max_q_len else tokens) * q_heads // self.num_heads
        if shared:
            _int32(shared, "shared")
            rows = (rows, tokens, q_heads, n, shared)
            _need(not window and 0 < shared <= width * self.page_tokens and
                  shared % self.page_tokens == 0,
                  "shared must be whole pages that a row of block_table can hold, without a window")
        size, ws, ws_at = self._sizes.get(rows), None, None
        if size is None:
            need = ct.c_size_t(0)
            if shared:
                _check(L.cg_int4_attention_shared_workspace(self._ref, a, shared, ct.byref(need)),
                       "cg_int4_attention_shared_workspace")
            else:
                _check(L.cg_int4_attention_workspace(self._ref, a, ct.byref(need)),
                       "cg_int4_attention_workspace")
            size = self._keep_size(rows, need.value)
        if size:
            # one per call, from the current stream's pool: calls on other
            # streams and captured graphs never share one
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
            ws_at = ws.data_ptr()
        with _Launch(dev.index) as s:
            if shared:
                st = L.cg_int4_attention_shared(self._ref, layer, a, shared, ws_at, size, s)
            else:
                st = L.cg_int4_attention(self._ref, layer, a, ws_at, size, s)
        _check(st, "cg_int4_attention")
        return out

    def _keep_size(self, key, size: int) -> int:
        if len(self._sizes) >= 1024:
            self._sizes.clear()
        self._sizes[key] = size
        return size

    def weigh(self, q, cu_q, kv_lens, block_table, weights=None, layer: int = 0, window: int = 0,
              sinks: int = 0, scale: float | None = None, max_q_len: int | None = None, out=None,
              stream=None):
        """Add the attention weights that the cached tokens get from the new tokens'
        queries, summed per KV head (cg_int4_weigh in include/cachegen.h), to
        ``weights`` (fp32 [requests, heads, n], a row of it per row of block_table, n at
        least every kv_lens[r]). The other arguments are those of attention, and so are the
        weights. The sums go to ``out`` (like weights), or to weights itself;
        without either a new tensor [requests, heads, pages of a row * page_tokens] is made of
        zeros. Elements behind a request's last token are not written: a row starts as
        zeros with its request. Returns what was written."""
        if stream is not None:
            return _on_stream(stream, self.weigh, q, cu_q, kv_lens, block_table, weights, layer, window,
                              sinks, scale, max_q_len, out)
        torch, dev, D = _torch, self.device, self.head_size
        shape = q.shape
        _need(len(shape) == 3, "q must be [tokens, q_heads, head_size]")
        _int32(layer, "layer")
        tokens, q_heads, _ = shape
        if q_heads <= 0 or q_heads % self.num_heads:
            raise ValueError(f"q_heads must be a multiple of {self.num_heads}")
        q_at, (qs0, qs1) = _bf16_rows(q, dev, (tokens, q_heads, D), "q", False)
        n, width, stride = _table(block_table, dev, "block_table")
        lens_at = _ints(kv_lens, dev, (n,), "kv_lens (one entry per row of block_table)")
        cu_at = _ints(cu_q, dev, (n + 1,), "cu_q")
        if out is None and weights is None:
            out = torch.zeros((n, self.num_heads, width * self.page_tokens), dtype=torch.float32, device=dev)
        elif out is None:
            out = weights
        _need(isinstance(out, torch.Tensor) and out.dim() == 3, "weights must be [requests, heads, tokens]")
        shape = (n, self.num_heads, out.shape[2])
        out_at, (os0, os1) = _floats(out, dev, shape, "out" if out is not weights else "weights", True)
        in_at = is0 = is1 = 0
        if weights is out:
            in_at, is0, is1 = out_at, os0, os1
        elif weights is not None:
            in_at, (is0, is1) = _floats(weights, dev, shape, "weights", False)
        try:
            a = _ATTENTION.pack(q_at, qs0, qs1, 0, 0, 0, cu_at, lens_at, block_table.data_ptr(), stride, width,
                                n, tokens, q_heads, max_q_len or 0, window, sinks,
                                D ** -0.5 if scale is None else scale)
            w = _WEIGHTS.pack(in_at, out_at, is0, is1, os0, os1, shape[2])
        except struct.error as e:
            raise ValueError(f"a number does not fit its type: {e}") from None
        L = _lib or load()
        key = (tokens, q_heads, max_q_len, n, width, shape[2])
        size = self._sizes.get(key)
        if size is None:
            need = ct.c_size_t(0)
            _check(L.cg_int4_weigh_workspace(self._ref, a, w, ct.byref(need)), "cg_int4_weigh_workspace")
            size = self._keep_size(key, need.value)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)   # one per call, as for attention
        with _Launch(dev.index) as s:
            st = L.cg_int4_weigh(self._ref, layer, a, w, ws.data_ptr(), size, s)
        _check(st, "cg_int4_weigh")
        return out

    def compact(self, kept, new_lens, lens, block_table, weights=None, layer: int = 0, stream=None) -> None:
        """Move the tokens that stay to the front of their request's pages
        (cg_int4_compact in include/cachegen.h): token kept[r, h, i] of request r's head
        h goes to place i < new_lens[r]. kept is int32 [requests, heads, budget] for one
        layer, or [layers, requests, heads, budget] for the layers from ``layer`` on,
        as choose_tokens gives it with new_lens. ``weights`` (fp32 [requests, heads, n], with
        layers where kept has them) move along, and what is behind becomes 0. The pages behind
        can then be given back with release_pages, once every layer has been compacted."""
        if stream is not None:
            return _on_stream(stream, self.compact, kept, new_lens, lens, block_table, weights, layer)
        torch, dev = _torch, self.device
        _need(isinstance(kept, torch.Tensor) and kept.dtype is torch.int32 and kept.device == dev and
              kept.dim() in (3, 4), f"kept must be an int32 tensor [requests, heads, budget] on {dev}, with or "
                                    f"without layers")
        shape = tuple(kept.shape)
        layers, budget = shape[0] if len(shape) == 4 else 1, shape[-1]
        n, width, stride = _table(block_table, dev, "block_table")
        _need(shape[-3:-1] == (n, self.num_heads), f"kept must be [requests, heads, budget] = [{n}, "
                                                   f"{self.num_heads}, budget], with or without layers")
        ks = kept.stride()
        _need(budget <= 1 or ks[-1] == 1 or kept.numel() == 0, "kept: entries of a row must be adjacent")
        ks = [s if m > 1 else 0 for s, m in zip(ks[:-1], shape)]
        lens_at, new_at = _ints(lens, dev, (n,), "lens"), _ints(new_lens, dev, (n,), "new_lens")
        w_at, wstr, w_width = 0, [0] * len(ks), 0
        if weights is not None:
            _need(isinstance(weights, torch.Tensor) and weights.dim() == len(shape), "weights must have kept's dimensions")
            w_width = weights.shape[-1]
            w_at, wstr = _floats(weights, dev, shape[:-1] + (w_width,), "weights", True)
            w_at = w_at or 256   # (an empty tensor has no address: lengths are still held against its width)
        if len(shape) == 3:
            ks, wstr = [0] + ks, [0] + wstr
        _int32(layer, "layer")
        try:
            c = _COMPACTION.pack(kept.data_ptr(), *ks, w_at, *wstr, w_width, budget, layers, n, lens_at,
                                 new_at, block_table.data_ptr(), stride, width)
        except struct.error as e:
            raise ValueError(f"a number does not fit its type: {e}") from None
        with _Launch(dev.index) as s:
            st = (_lib or load()).cg_int4_compact(self._ref, layer, c, s)
        _check(st, "cg_int4_compact")

    def check(self):
        """Wait for the current stream; raise the first error that the GPU
        found in this cache's calls since the last check. It is read and cleared
        in one step: what calls on other streams meet later stays for the next
        check."""
        import torch
        with torch.cuda.device(self.device):
            result = torch.empty(16, dtype=torch.uint8, device=self.device)
            _check(load().cg_int4_take_error(self._ref, result.data_ptr(), _stream_handle()),
                   "cg_int4_take_error")
            st, _ = cg_last_device_error(None, result)
        _check(st, "Int4Cache (device)")
