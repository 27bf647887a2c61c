"""Python binding of libmla: MLA latent-KV decode on B200 (sm_100a).

Argument marshalling only: every function here forwards torch tensors (device memory owned
by the caller) and integers to the C ABI of the same name in ``include/mla.h`` and raises
``MlaError`` on a non-OK status.  All computation happens in the library's CUDA kernels;
there is no fallback: importing works without a GPU, but calling anything needs the built
``libmla.so`` (``python -m mla_latent_kv_24_b200.build``) and a CUDA device.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

__all__ = [
    "MlaError", "mla_dims", "make_dims", "load", "LIB_PATH", "STATUS",
    "mla_cache_append", "mla_decode_workspace_size", "mla_decode_absorbed",
    "gqla_expand_cache", "gqla_decode_workspace_size", "gqla_decode_grouped",
    "mla_get_device_status", "mla_last_error_string", "mla_version", "mla_set_profile_events",
    "mla_decode_absorbed_noalloc", "NOALLOC_SCRATCH_BYTES", "EXPORTED_SYMBOLS", "mla_select_path",
    "mla_prefill_workspace_size", "mla_prefill_expanded", "gqla_expand_tokens", "mla_debug_decode_fault",
    "mla_decode_tree_workspace_size", "mla_decode_tree", "mla_decode_window_workspace_size", "mla_decode_window",
    "gqla_decode_window_workspace_size", "gqla_decode_window", "mla_cache_append_slots", "mla_cache_reserve",
    "mla_cache_fork", "mla_cache_release", "mla_cache_accept", "MAX_TREE_NODES",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla.so")

STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
          4: "MLA_ERR_CUDA", 5: "MLA_ERR_DEVICE_BOUNDS", 6: "MLA_ERR_TIMEOUT", 7: "MLA_ERR_NO_PAGES"}
MLA_BF16, MLA_FP32 = 0, 1

EXPORTED_SYMBOLS = ["mla_cache_append", "mla_decode_workspace_size", "mla_decode_absorbed",
                    "gqla_expand_cache", "gqla_decode_workspace_size", "gqla_decode_grouped",
                    "mla_get_device_status", "mla_last_error_string", "mla_version", "mla_set_profile_events",
                    "mla_decode_absorbed_noalloc", "mla_select_path", "mla_prefill_workspace_size",
                    "mla_prefill_expanded", "gqla_expand_tokens", "mla_debug_decode_fault",
                    "mla_decode_tree_workspace_size", "mla_decode_tree", "mla_decode_window_workspace_size",
                    "mla_decode_window", "gqla_decode_window_workspace_size", "gqla_decode_window",
                    "mla_cache_append_slots", "mla_cache_reserve", "mla_cache_fork", "mla_cache_release",
                    "mla_cache_accept"]
NOALLOC_SCRATCH_BYTES = 32 << 20
MAX_TREE_NODES = 64


class MlaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class mla_dims(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("heads_per_group", ctypes.c_int32), ("d_c", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("d_nope", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("rope_base", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


def make_dims(n_heads=128, heads_per_group=1, d_c=512, d_rope=64, d_nope=128, d_v=128, page_size=64,
              softmax_scale=0.0, rope_base=10000.0, dtype="bf16") -> mla_dims:
    return mla_dims(n_heads, heads_per_group, d_c, d_rope, d_nope, d_v, page_size, softmax_scale, rope_base,
                    MLA_BF16 if dtype == "bf16" else MLA_FP32)


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_S = ctypes.c_size_t


def load() -> ctypes.CDLL:
    """Loads libmla.so (once).  Raises ImportError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m mla_latent_kv_24_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    D = ctypes.POINTER(mla_dims)
    sig = {
        "mla_cache_append": [D, _P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _P],
        "mla_decode_workspace_size": [D, _I, _I, _P, ctypes.POINTER(_S)],
        "mla_decode_absorbed": [D, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _S, _P],
        "gqla_expand_cache": [D, _P, _P, _P, _P, _I, _I, _P, _P],
        "gqla_expand_tokens": [D, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _P],
        "gqla_decode_workspace_size": [D, _I, _I, _P, ctypes.POINTER(_S)],
        "gqla_decode_grouped": [D, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _S, _P],
        "mla_get_device_status": [_P],
        "mla_last_error_string": [],
        "mla_version": [],
        "mla_set_profile_events": [_P, _P],
        "mla_decode_absorbed_noalloc": [D, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P],
        "mla_select_path": [D, _I, _I, _P, ctypes.c_double, ctypes.c_double, _I, ctypes.POINTER(ctypes.c_int),
                            ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)],
        "mla_prefill_workspace_size": [D, _I, _I, _P, ctypes.POINTER(_S)],
        "mla_prefill_expanded": [D, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _S, _P],
        "mla_debug_decode_fault": [_I, ctypes.c_uint32],
        "mla_decode_tree_workspace_size": [D, _I, _I, _P, _P, ctypes.POINTER(_S)],
        "mla_decode_tree": [D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _S, _P],
        "mla_decode_window_workspace_size": [D, _I, _I, _I, _I, _P, ctypes.POINTER(_S)],
        "mla_decode_window": [D, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _S, _P],
        "gqla_decode_window_workspace_size": [D, _I, _I, _I, _I, _P, ctypes.POINTER(_S)],
        "gqla_decode_window": [D, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _S, _P],
        "mla_cache_append_slots": [D, _P, _I, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _P],
        "mla_cache_reserve": [D, _P, _P, _P, _I, _I, _P, _I, _P],
        "mla_cache_fork": [D, _P, _P, _I, _P, _P, _I, _I, _P, _I, _P, _P, _I, _P],
        "mla_cache_release": [D, _P, _P, _P, _I, _P, _P, _I, _I, _P, _I, _P],
        "mla_cache_accept": [D, _P, _P, _P, _P, _I, _P, _P, _I, _I, _P, _I, _P, _P, _I, _P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_char_p if name == "mla_last_error_string" else ctypes.c_int
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise MlaError(status, load().mla_last_error_string().decode())


def _dev(t) -> Optional[int]:
    """Device address of a CUDA tensor (None stays NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # 0.1 us; the Stream object costs 3
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _host_i32(x: Sequence[int]):
    a = np.ascontiguousarray(np.asarray(x, dtype=np.int32))
    return a, a.ctypes.data_as(ctypes.c_void_p)


def mla_cache_append(dims, h, hidden, W_dkv, W_kr, req_idx, positions, n_tok, page_table, batch, max_pages,
                     n_pages_total, latent_cache, stream=None) -> None:
    _check(load().mla_cache_append(ctypes.byref(dims), _dev(h), hidden, _dev(W_dkv), _dev(W_kr), _dev(req_idx),
                                   _dev(positions), n_tok, _dev(page_table), batch, max_pages, n_pages_total,
                                   _dev(latent_cache), _stream(stream)))


def mla_decode_workspace_size(dims, batch, s_q, seq_lens_host) -> int:
    arr, p = _host_i32(seq_lens_host)
    out = _S(0)
    _check(load().mla_decode_workspace_size(ctypes.byref(dims), batch, s_q, p, ctypes.byref(out)))
    return out.value


def gqla_decode_workspace_size(dims, batch, s_q, seq_lens_host) -> int:
    arr, p = _host_i32(seq_lens_host)
    out = _S(0)
    _check(load().gqla_decode_workspace_size(ctypes.byref(dims), batch, s_q, p, ctypes.byref(out)))
    return out.value


def mla_decode_absorbed(dims, q, W_uk, W_uv, latent_cache, page_table, seq_lens, seq_lens_host, batch, s_q,
                        max_pages, n_pages_total, out, workspace, workspace_bytes=None, stream=None) -> None:
    arr, p = _host_i32(seq_lens_host)
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().mla_decode_absorbed(ctypes.byref(dims), _dev(q), _dev(W_uk), _dev(W_uv), _dev(latent_cache),
                                      _dev(page_table), _dev(seq_lens), p, batch, s_q, max_pages, n_pages_total,
                                      _dev(out), _dev(workspace), nbytes, _stream(stream)))


def gqla_expand_cache(dims, W_uk, W_uv, latent_cache, page_ids, n_ids, n_pages_total, expanded_cache,
                      stream=None) -> None:
    _check(load().gqla_expand_cache(ctypes.byref(dims), _dev(W_uk), _dev(W_uv), _dev(latent_cache), _dev(page_ids),
                                    n_ids, n_pages_total, _dev(expanded_cache), _stream(stream)))


def gqla_expand_tokens(dims, W_uk, W_uv, latent_cache, req_idx, positions, n_tok, page_table, batch, max_pages,
                       n_pages_total, expanded_cache, stream=None) -> None:
    _check(load().gqla_expand_tokens(ctypes.byref(dims), _dev(W_uk), _dev(W_uv), _dev(latent_cache), _dev(req_idx),
                                     _dev(positions), n_tok, _dev(page_table), batch, max_pages, n_pages_total,
                                     _dev(expanded_cache), _stream(stream)))


def gqla_decode_grouped(dims, q, expanded_cache, latent_cache, page_table, seq_lens, seq_lens_host, batch, s_q,
                        max_pages, n_pages_total, out, workspace, workspace_bytes=None, stream=None) -> None:
    arr, p = _host_i32(seq_lens_host)
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().gqla_decode_grouped(ctypes.byref(dims), _dev(q), _dev(expanded_cache), _dev(latent_cache),
                                      _dev(page_table), _dev(seq_lens), p, batch, s_q, max_pages, n_pages_total,
                                      _dev(out), _dev(workspace), nbytes, _stream(stream)))


def mla_get_device_status(stream=None) -> None:
    _check(load().mla_get_device_status(_stream(stream)))


def mla_last_error_string() -> str:
    return load().mla_last_error_string().decode()


def mla_version() -> int:
    return int(load().mla_version())


def mla_set_profile_events(start=None, stop=None) -> None:
    """Records torch.cuda.Event `start`/`stop` around the main attention kernel of later decode
    calls on this thread (None, None turns it off).  The events must already exist: record
    each once before passing it."""
    s = None if start is None else ctypes.c_void_p(start.cuda_event)
    e = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    _check(load().mla_set_profile_events(s, e))


def mla_decode_absorbed_noalloc(dims, q, W_uk, W_uv, latent_cache, page_table, seq_lens, seq_lens_host, batch, s_q,
                                max_pages, n_pages_total, out, stream=None) -> None:
    """mla_decode_absorbed without a workspace argument, for callers that cannot allocate device
    memory: the library's own static scratch (NOALLOC_SCRATCH_BYTES per device) is used.  Calls
    that overlap on the GPU race on that scratch; batches that need more raise MlaError."""
    arr, p = _host_i32(seq_lens_host)
    _check(load().mla_decode_absorbed_noalloc(ctypes.byref(dims), _dev(q), _dev(W_uk), _dev(W_uv), _dev(latent_cache),
                                              _dev(page_table), _dev(seq_lens), p, batch, s_q, max_pages,
                                              n_pages_total, _dev(out), _stream(stream)))


def mla_select_path(dims, batch, s_q, seq_lens_host, hbm_bytes_per_s, flops_per_s, tp=1):
    """Roofline choice between the two decoding paths (host arithmetic only, no GPU needed).
    Returns ("absorbed" | "grouped", modelled seconds of the absorbed path, of the grouped path)."""
    lens, lp = _host_i32(seq_lens_host)
    path = ctypes.c_int(0)
    ta, tg = ctypes.c_double(0.0), ctypes.c_double(0.0)
    _check(load().mla_select_path(ctypes.byref(dims), batch, s_q, lp, float(hbm_bytes_per_s), float(flops_per_s), tp,
                                  ctypes.byref(path), ctypes.byref(ta), ctypes.byref(tg)))
    return ("grouped" if path.value == 1 else "absorbed"), ta.value, tg.value


def mla_prefill_workspace_size(dims, batch, n_q, seq_lens_host) -> int:
    arr, p = _host_i32(seq_lens_host)
    n = _S(0)
    _check(load().mla_prefill_workspace_size(ctypes.byref(dims), batch, n_q, p, ctypes.byref(n)))
    return n.value


def mla_prefill_expanded(dims, q, expanded_cache, latent_cache, page_table, seq_lens, seq_lens_host, batch, n_q,
                         max_pages, n_pages_total, out, workspace, workspace_bytes=None, stream=None) -> None:
    arr, p = _host_i32(seq_lens_host)
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().mla_prefill_expanded(ctypes.byref(dims), _dev(q), _dev(expanded_cache), _dev(latent_cache),
                                       _dev(page_table), _dev(seq_lens), p, batch, n_q, max_pages, n_pages_total,
                                       _dev(out), _dev(workspace), nbytes, _stream(stream)))


def mla_debug_decode_fault(withhold_step: int, wait_us: int = 0) -> None:
    """Test hook: later tensor-core absorbed decodes on this thread withhold the completion signal
    of pipeline step `withhold_step` (-1 restores normal operation) and give up every device wait
    after `wait_us` microseconds (0: the 2 s default).  See include/mla.h."""
    _check(load().mla_debug_decode_fault(withhold_step, wait_us))


# ---------------------------------------------------------------------------------------
# Trees, windows and the page pool.  The arrays these calls index by come from several of the
# caller's structures, so their types, sizes and device are checked here: a short or narrow one
# would be read past its end.
# ---------------------------------------------------------------------------------------
_torch = None   # the module, kept: an import statement costs 0.1 us of a call
_INT = None     # torch.int32, the type of every index array, once torch is there


def _here() -> int:
    """The current device; one that no tensor is on while CUDA has not been used."""
    global _torch, _INT
    if _torch is None:
        import torch
        _torch, _INT = torch, torch.int32
    return _torch._C._cuda_getDevice() if _torch.cuda.is_initialized() else -2


def _stream_on(stream, here) -> Optional[int]:
    """_stream for a caller that knows the current device."""
    if stream is None and here >= 0:
        raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(here)
    return _stream(stream)


def _elt(dims):
    """The type of a call's float tensors."""
    return _torch.float32 if dims.dtype == MLA_FP32 else _torch.bfloat16


def _arr(name, t, dtype, n, here, optional=False) -> Optional[int]:
    """Device address of a contiguous tensor of at least n elements of `dtype` on device `here`."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is None")
    if t.get_device() != here or t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        _dev(t)
        if t.get_device() != here:
            raise ValueError(f"{name} is on {t.device}, not on the current device")
        if t.dtype is not dtype:
            raise ValueError(f"{name} holds {t.dtype}, expected {dtype}")
        raise ValueError(f"{name} has {t.numel()} elements, expected at least {n}")
    return t.data_ptr()


def _host_lens(name, x, n):
    """(array that keeps the memory, address) of a host int32 array of at least n elements."""
    a = x if type(x) is np.ndarray and x.dtype == np.int32 and x.flags.c_contiguous else \
        np.ascontiguousarray(np.asarray(x, dtype=np.int32))
    if a.size < n:
        raise ValueError(f"{name} has {a.size} elements, expected at least {n}")
    try:
        return a, ctypes.addressof(ctypes.c_char.from_buffer(a))   # a third of the time of a.ctypes.data
    except (TypeError, ValueError):                                # read-only, or empty
        return a, a.ctypes.data


def _decode_view_args(dims, q, s_q, cache, n_pages_total, batch, max_pages, page_table, seq_lens, out, here):
    e = _elt(dims)
    rows = batch * s_q * dims.n_heads
    return e, (_arr("q", q, e, rows * (dims.d_nope + dims.d_rope), here),
               _arr("latent_cache", cache, e, n_pages_total * dims.page_size * (dims.d_c + dims.d_rope), here),
               _arr("page_table", page_table, _INT, batch * max_pages, here), _arr("seq_lens", seq_lens, _INT, batch, here),
               _arr("out", out, e, rows * dims.d_v, here))


def _weights(dims, e, W_uk, W_uv, here):
    g = dims.n_heads // max(1, dims.heads_per_group)
    return _arr("W_uk", W_uk, e, g * dims.d_nope * dims.d_c, here), _arr("W_uv", W_uv, e, g * dims.d_v * dims.d_c, here)


def _workspace(ws, nbytes, here):
    have = ws.numel() * ws.itemsize
    return _arr("workspace", ws, ws.dtype, 0, here), have if nbytes is None else min(nbytes, have)


def mla_decode_tree_workspace_size(dims, batch, max_nodes, seq_lens_host, n_nodes_host) -> int:
    lens, lp = _host_lens("seq_lens_host", seq_lens_host, batch)
    nodes, np_ = _host_lens("n_nodes_host", n_nodes_host, batch)
    out = _S(0)
    _check(load().mla_decode_tree_workspace_size(ctypes.byref(dims), batch, max_nodes, lp, np_, ctypes.byref(out)))
    return out.value


def mla_decode_tree(dims, q, W_uk, W_uv, latent_cache, page_table, seq_lens, n_nodes, seq_lens_host, n_nodes_host,
                    depths, tree_mask, batch, max_nodes, max_pages, n_pages_total, out, workspace,
                    workspace_bytes=None, stream=None) -> None:
    """Attention of a tree of up to 64 drafted tokens per request over the latent cache.  `tree_mask` is an
    int64 (or uint64) tensor of bit masks; see include/mla.h."""
    lens, lp = _host_lens("seq_lens_host", seq_lens_host, batch)
    nodes, np_ = _host_lens("n_nodes_host", n_nodes_host, batch)
    here = _here()
    e, (qp, cp, tp, sp, op) = _decode_view_args(dims, q, max_nodes, latent_cache, n_pages_total, batch, max_pages,
                                                page_table, seq_lens, out, here)
    uk, uv = _weights(dims, e, W_uk, W_uv, here)
    ws, nbytes = _workspace(workspace, workspace_bytes, here)
    mask_type = _torch.uint64 if tree_mask is not None and tree_mask.dtype is _torch.uint64 else _torch.int64
    _check(load().mla_decode_tree(ctypes.byref(dims), qp, uk, uv, cp, tp, sp,
                                  _arr("n_nodes", n_nodes, _INT, batch, here), lp, np_,
                                  _arr("depths", depths, _INT, batch * max_nodes, here),
                                  _arr("tree_mask", tree_mask, mask_type, batch * max_nodes, here), batch, max_nodes, max_pages,
                                  n_pages_total, op, ws, nbytes, _stream_on(stream, here)))


def mla_decode_window_workspace_size(dims, batch, s_q, sinks, window, seq_lens_host) -> int:
    lens, lp = _host_lens("seq_lens_host", seq_lens_host, batch)
    out = _S(0)
    _check(load().mla_decode_window_workspace_size(ctypes.byref(dims), batch, s_q, sinks, window, lp,
                                                   ctypes.byref(out)))
    return out.value


def mla_decode_window(dims, q, W_uk, W_uv, latent_cache, page_table, seq_lens, seq_lens_host, batch, s_q, sinks,
                      window, max_pages, n_pages_total, out, workspace, workspace_bytes=None, stream=None) -> None:
    lens, lp = _host_lens("seq_lens_host", seq_lens_host, batch)
    here = _here()
    e, (qp, cp, tp, sp, op) = _decode_view_args(dims, q, s_q, latent_cache, n_pages_total, batch, max_pages,
                                                page_table, seq_lens, out, here)
    uk, uv = _weights(dims, e, W_uk, W_uv, here)
    ws, nbytes = _workspace(workspace, workspace_bytes, here)
    _check(load().mla_decode_window(ctypes.byref(dims), qp, uk, uv, cp, tp, sp, lp, batch, s_q, sinks, window,
                                    max_pages, n_pages_total, op, ws, nbytes, _stream_on(stream, here)))


def gqla_decode_window_workspace_size(dims, batch, s_q, sinks, window, seq_lens_host) -> int:
    lens, lp = _host_lens("seq_lens_host", seq_lens_host, batch)
    out = _S(0)
    _check(load().gqla_decode_window_workspace_size(ctypes.byref(dims), batch, s_q, sinks, window, lp,
                                                    ctypes.byref(out)))
    return out.value


def gqla_decode_window(dims, q, expanded_cache, latent_cache, page_table, seq_lens, seq_lens_host, batch, s_q, sinks,
                       window, max_pages, n_pages_total, out, workspace, workspace_bytes=None, stream=None) -> None:
    lens, lp = _host_lens("seq_lens_host", seq_lens_host, batch)
    here = _here()
    e, (qp, cp, tp, sp, op) = _decode_view_args(dims, q, s_q, latent_cache, n_pages_total, batch, max_pages,
                                                page_table, seq_lens, out, here)
    g = dims.n_heads // max(1, dims.heads_per_group)
    ep = _arr("expanded_cache", expanded_cache, e, n_pages_total * g * dims.page_size * (dims.d_nope + dims.d_v), here)
    ws, nbytes = _workspace(workspace, workspace_bytes, here)
    _check(load().gqla_decode_window(ctypes.byref(dims), qp, ep, cp, tp, sp, lp, batch, s_q, sinks, window, max_pages,
                                     n_pages_total, op, ws, nbytes, _stream_on(stream, here)))


def mla_cache_append_slots(dims, h, hidden, W_dkv, W_kr, req_idx, slots, positions, n_tok, page_table, batch,
                           max_pages, n_pages_total, latent_cache, stream=None) -> None:
    row, here = dims.d_c + dims.d_rope, _here()
    e = _elt(dims)
    _check(load().mla_cache_append_slots(
        ctypes.byref(dims), _arr("h", h, e, n_tok * hidden, here), hidden,
        _arr("W_dkv", W_dkv, e, dims.d_c * hidden, here, True),
        _arr("W_kr", W_kr, e, dims.d_rope * hidden, here, True), _arr("req_idx", req_idx, _INT, n_tok, here),
        _arr("slots", slots, _INT, n_tok, here), _arr("positions", positions, _INT, n_tok, here), n_tok,
        _arr("page_table", page_table, _INT, batch * max_pages, here), batch, max_pages, n_pages_total,
        _arr("latent_cache", latent_cache, e, n_pages_total * dims.page_size * row, here), _stream_on(stream, here)))


def _pool_args(seq_lens, page_table, batch, max_pages, page_refs, n_pages_total, here, refs_optional=False):
    return (_arr("seq_lens", seq_lens, _INT, batch, here), _arr("page_table", page_table, _INT, batch * max_pages, here),
            _arr("page_refs", page_refs, _INT, n_pages_total, here, refs_optional))


def _cache_args(dims, latent_cache, expanded_cache, n_layers, n_pages_total, here):
    e = _elt(dims)
    rows = n_layers * n_pages_total * dims.page_size
    g = dims.n_heads // max(1, dims.heads_per_group)
    return (_arr("latent_cache", latent_cache, e, rows * (dims.d_c + dims.d_rope), here, True),
            _arr("expanded_cache", expanded_cache, e, rows * g * (dims.d_nope + dims.d_v), here, True))


def mla_cache_reserve(dims, new_lens, seq_lens, page_table, batch, max_pages, page_refs, n_pages_total,
                      stream=None) -> None:
    here = _here()
    s, t, r = _pool_args(seq_lens, page_table, batch, max_pages, page_refs, n_pages_total, here)
    _check(load().mla_cache_reserve(ctypes.byref(dims), _arr("new_lens", new_lens, _INT, batch, here), s, t, batch,
                                    max_pages, r, n_pages_total, _stream_on(stream, here)))


def mla_cache_fork(dims, src_req, dst_req, n_fork, seq_lens, page_table, batch, max_pages, page_refs, n_pages_total,
                   latent_cache, expanded_cache, n_layers, stream=None) -> None:
    here = _here()
    s, t, r = _pool_args(seq_lens, page_table, batch, max_pages, page_refs, n_pages_total, here)
    lat, exp = _cache_args(dims, latent_cache, expanded_cache, n_layers, n_pages_total, here)
    _check(load().mla_cache_fork(ctypes.byref(dims), _arr("src_req", src_req, _INT, n_fork, here),
                                 _arr("dst_req", dst_req, _INT, n_fork, here), n_fork, s, t, batch, max_pages, r,
                                 n_pages_total, lat, exp, n_layers, _stream_on(stream, here)))


def mla_cache_release(dims, req_idx, first_page, last_page, n_req, seq_lens, page_table, batch, max_pages, page_refs,
                      n_pages_total, stream=None) -> None:
    here = _here()
    s, t, r = _pool_args(seq_lens, page_table, batch, max_pages, page_refs, n_pages_total, here)
    _check(load().mla_cache_release(ctypes.byref(dims), _arr("req_idx", req_idx, _INT, n_req, here),
                                    _arr("first_page", first_page, _INT, n_req, here, True),
                                    _arr("last_page", last_page, _INT, n_req, here, True), n_req, s, t, batch, max_pages,
                                    r, n_pages_total, _stream_on(stream, here)))


def mla_cache_accept(dims, ctx_lens, n_nodes, accepted, n_accepted, max_nodes, seq_lens, page_table, batch, max_pages,
                     page_refs, n_pages_total, latent_cache, expanded_cache, n_layers, stream=None) -> None:
    here = _here()
    s, t, r = _pool_args(seq_lens, page_table, batch, max_pages, page_refs, n_pages_total, here, True)
    lat, exp = _cache_args(dims, latent_cache, expanded_cache, n_layers, n_pages_total, here)
    _check(load().mla_cache_accept(ctypes.byref(dims), _arr("ctx_lens", ctx_lens, _INT, batch, here),
                                   _arr("n_nodes", n_nodes, _INT, batch, here),
                                   _arr("accepted", accepted, _INT, batch * max_nodes, here),
                                   _arr("n_accepted", n_accepted, _INT, batch, here), max_nodes, s, t, batch, max_pages, r,
                                   n_pages_total, lat, exp, n_layers, _stream_on(stream, here)))
