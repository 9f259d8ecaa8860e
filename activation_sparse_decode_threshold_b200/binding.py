"""Thin Python binding of libpi_ffn.so (include/pi_ffn.h).

Argument marshalling only: every function here has the name of the C entry
point it calls, turns torch tensors into device/host pointers, and raises
``PiError`` on a non-OK status (the calls of the attention half do so in C++,
csrc/pi_torch.cpp).  Every step of the sparse FFN runs in the
library's CUDA kernels; nothing here computes.  Loading fails loudly when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpi_ffn.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "pi_ffn.h")

PI_OK, PI_ERR_INVALID_ARG, PI_ERR_UNSUPPORTED, PI_ERR_OOM = 0, 1, 2, 3
PI_ERR_CUDA, PI_ERR_TIMEOUT, PI_ERR_DEVICE_CHECK, PI_ERR_NOT_LOADED = 4, 5, 6, 7
STATUS = {0: "PI_OK", 1: "PI_ERR_INVALID_ARG", 2: "PI_ERR_UNSUPPORTED", 3: "PI_ERR_OOM",
          4: "PI_ERR_CUDA", 5: "PI_ERR_TIMEOUT", 6: "PI_ERR_DEVICE_CHECK", 7: "PI_ERR_NOT_LOADED"}
ACT = {"relu": 0, "reglu": 1, "drelu": 2}
DTYPE = {"f32": 0, "f16": 1, "bf16": 2, "int4g32": 3, "i8row": 4}
PI_DEBUG_STALL_BARRIER = 1
PI_DEBUG_STALL_PREFILL = 2
PI_DEBUG_STALL_T_POLL = 8


class PiError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class pi_ffn_desc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("d_ff", ctypes.c_int),
                ("rank", ctypes.c_int), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int),
                ("act", ctypes.c_int), ("w_dtype", ctypes.c_int), ("pred_dtype", ctypes.c_int),
                ("n_strips", ctypes.c_int), ("threshold", ctypes.c_float), ("eps", ctypes.c_float),
                ("device", ctypes.c_int)]


class pi_expert_weights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("U", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("s_U", ctypes.c_void_p), ("s_V", ctypes.c_void_p)]


class pi_attn_desc(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("cache_dtype", ctypes.c_int), ("page_size", ctypes.c_int), ("layout", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("rotary_pairs", ctypes.c_int), ("rope_theta", ctypes.c_float),
                ("norm_eps", ctypes.c_float), ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("window", ctypes.c_int), ("device", ctypes.c_int)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it was never built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m activation_sparse_decode_threshold_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, ip, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        sigs = {
            "pi_ffn_create": [ctypes.POINTER(pi_ffn_desc), ctypes.POINTER(vp)],
            "pi_ffn_load_layer": [vp, ip, ctypes.POINTER(pi_expert_weights), vp, vp, vp],
            "pi_neuron_table": [vp, ip, ip, vp],
            "pi_strip_offsets": [vp, vp, ctypes.POINTER(ip)],
            "pi_predict": [vp, ip, ip, vp, vp, vp, vp, vp],
            "pi_sparse_ffn_decode": [vp, ip, ip, vp, vp, vp, vp, vp],
            "pi_sparse_ffn_decode_host": [vp, ip, ip, vp, vp, vp],
            "pi_sparse_ffn_decode_batch": [vp, ip, ip, ip, vp, vp, vp, vp, vp],
            "pi_sparse_ffn_decode_partial": [vp, ip, vp, vp, vp, vp, vp],
            "pi_residual_add": [vp, vp, vp, vp],
            "pi_ffn_set_hot_neurons": [vp, ip],
            "pi_dense_ffn_prefill": [vp, ip, ip, ip, vp, vp],
            "pi_sync": [vp, vp],
            "pi_debug_set": [vp, ip, ctypes.c_double],
            "pi_debug_phase_times": [vp, vp],
            "pi_predict_noalloc": [ip, ip, ip, ip, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp],
            "pi_int4_create": [ip, ip, vp, vp, ip, vp, ctypes.POINTER(vp)],
            "pi_int4_matvec": [vp, ip, ip, vp, i64, vp, ip, vp, i64, ctypes.c_float, vp],
            "pi_attn_create": [ctypes.POINTER(pi_attn_desc), ctypes.POINTER(vp)],
            "pi_attn_sync": [vp, vp],
            "pi_kv_append": [vp, vp, vp, ip, vp, vp, ip, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp],
            "pi_kv_read": [vp, vp, vp, ip, vp, vp, ip, vp, vp, vp],
            "pi_paged_attention": [vp, vp, vp, vp, ip, vp, i64, vp, i64, vp, vp],
        }
        for name, args in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.pi_last_error.argtypes = []
        L.pi_last_error.restype = ctypes.c_char_p
        for name in ("pi_ffn_destroy", "pi_int4_destroy", "pi_attn_destroy"):
            getattr(L, name).argtypes = [vp]
            getattr(L, name).restype = None
        _lib = L
    return _lib


def header_symbols() -> list[str]:
    """Entry points declared in include/pi_ffn.h."""
    with open(HEADER) as f:
        return re.findall(r"^PI_API\s+[^(]*?\b(pi_\w+)\s*\(", f.read(), flags=re.M)


def _check(st: int, where: str):
    if st != PI_OK:
        raise PiError(st, where, lib().pi_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def pi_last_error() -> str:
    return lib().pi_last_error().decode()


def pi_ffn_create(n_layers, d_model, d_ff, rank, act="reglu", w_dtype="f16", pred_dtype="f16",
                  n_experts=1, top_k=1, n_strips=0, threshold=0.0, eps=1e-6, device=0) -> int:
    desc = pi_ffn_desc(n_layers, d_model, d_ff, rank, n_experts, top_k, ACT[act], DTYPE[w_dtype],
                       DTYPE[pred_dtype], n_strips, threshold, eps, device)
    h = ctypes.c_void_p()
    _check(lib().pi_ffn_create(ctypes.byref(desc), ctypes.byref(h)), "pi_ffn_create")
    return h.value


def pi_ffn_destroy(h: int):
    if h:
        lib().pi_ffn_destroy(h)


def pi_ffn_load_layer(h, layer, experts, router=None, freq=None, stream=None):
    """`experts`: list of objects with attributes w_gate, w_up, w_down, s_gate,
    s_up, s_down, c (bias), U, V, sU, sV (device tensors, None where absent).
    `freq`: host float32 array (n_experts x F) or None."""
    import numpy as np
    arr = (pi_expert_weights * len(experts))()
    for i, e in enumerate(experts):
        arr[i] = pi_expert_weights(_ptr(e.w_gate), _ptr(e.w_up), _ptr(e.w_down),
                                   _ptr(getattr(e, "s_gate", None)), _ptr(getattr(e, "s_up", None)),
                                   _ptr(getattr(e, "s_down", None)), _ptr(e.c), _ptr(e.U), _ptr(e.V),
                                   _ptr(getattr(e, "sU", None)), _ptr(getattr(e, "sV", None)))
    fq = None
    if freq is not None:
        fq = np.ascontiguousarray(np.asarray(freq, np.float32))
    _check(lib().pi_ffn_load_layer(h, layer, arr, _ptr(router),
                                   None if fq is None else fq.ctypes.data, _stream(stream)),
           "pi_ffn_load_layer")


def pi_ffn_set_hot_neurons(h, hot_per_strip: int):
    _check(lib().pi_ffn_set_hot_neurons(h, hot_per_strip), "pi_ffn_set_hot_neurons")


def pi_neuron_table(h, layer, expert, F):
    import numpy as np
    perm = np.empty(F, np.int32)
    _check(lib().pi_neuron_table(h, layer, expert, perm.ctypes.data), "pi_neuron_table")
    return perm


def pi_strip_offsets(h):
    import numpy as np
    n = ctypes.c_int()
    _check(lib().pi_strip_offsets(h, None, ctypes.byref(n)), "pi_strip_offsets")
    off = np.empty(n.value + 1, np.int32)
    _check(lib().pi_strip_offsets(h, off.ctypes.data, None), "pi_strip_offsets")
    return off


def pi_predict(h, layer, expert, x, idx, count, z=None, stream=None):
    _check(lib().pi_predict(h, layer, expert, _ptr(x), _ptr(idx), _ptr(count), _ptr(z),
                            _stream(stream)), "pi_predict")


def pi_sparse_ffn_decode(h, layer_begin, layer_end, resid, trace=None, stats=None, masks=None,
                         stream=None):
    _check(lib().pi_sparse_ffn_decode(h, layer_begin, layer_end, _ptr(resid), _ptr(trace),
                                      _ptr(stats), _ptr(masks), _stream(stream)),
           "pi_sparse_ffn_decode")


def pi_sparse_ffn_decode_batch(h, layer_begin, layer_end, resid, trace=None, stats=None, masks=None,
                               stream=None):
    """`resid`: device float32 tensor [n_tokens x d] (n_tokens = resid.shape[0])."""
    _check(lib().pi_sparse_ffn_decode_batch(h, layer_begin, layer_end, int(resid.shape[0]), _ptr(resid),
                                            _ptr(trace), _ptr(stats), _ptr(masks), _stream(stream)),
           "pi_sparse_ffn_decode_batch")


def pi_sparse_ffn_decode_partial(h, layer, resid, y, stats=None, masks=None, stream=None):
    _check(lib().pi_sparse_ffn_decode_partial(h, layer, _ptr(resid), _ptr(y), _ptr(stats), _ptr(masks),
                                              _stream(stream)), "pi_sparse_ffn_decode_partial")


def pi_residual_add(h, resid, y, stream=None):
    _check(lib().pi_residual_add(h, _ptr(resid), _ptr(y), _stream(stream)), "pi_residual_add")


def pi_sparse_ffn_decode_host(h, layer_begin, layer_end, resid_in, resid_out, stream=None):
    """resid_in / resid_out: host (ideally pinned) float32 tensors of d entries."""
    _check(lib().pi_sparse_ffn_decode_host(h, layer_begin, layer_end, _ptr(resid_in),
                                           _ptr(resid_out), _stream(stream)),
           "pi_sparse_ffn_decode_host")


def pi_dense_ffn_prefill(h, layer_begin, layer_end, n_tokens, resid, stream=None):
    _check(lib().pi_dense_ffn_prefill(h, layer_begin, layer_end, n_tokens, _ptr(resid),
                                      _stream(stream)), "pi_dense_ffn_prefill")


def pi_sync(h, stream=None) -> int:
    """Returns the status (does not raise), so callers can test for timeouts."""
    return lib().pi_sync(h, _stream(stream))


def pi_debug_set(h, flags: int, wait_limit_s: float):
    _check(lib().pi_debug_set(h, flags, wait_limit_s), "pi_debug_set")


def pi_debug_phase_times(h, times=None):
    _check(lib().pi_debug_phase_times(h, _ptr(times)), "pi_debug_phase_times")


def pi_predict_noalloc(d_model, d_ff, rank, pred_dtype, threshold, V, U, bias, x, idx, count, z=None,
                       stream=None):
    """Predictor on caller-owned weights (original order) with no device allocation."""
    _check(lib().pi_predict_noalloc(d_model, d_ff, rank, DTYPE[pred_dtype], threshold, _ptr(V), _ptr(U),
                                    _ptr(bias), _ptr(x), _ptr(idx), _ptr(count), _ptr(z), _stream(stream)),
           "pi_predict_noalloc")


# ---------------------------------------------------------------------------
# The attention half of a decode layer.  Shapes, row distances and types come
# from the tensors, so these wrappers check that the tensors are what the C
# entry point will take them for; a mismatch raises PI_ERR_INVALID_ARG.
# ---------------------------------------------------------------------------
KV_LAYOUT = {"hnd": 0, "nhd": 1}
_desc: dict = {}     # handle -> what the checks need of it
_native_module = None
EXT_PATH = os.path.join(HERE, "_pi_torch.so")


def _native():
    """The native part (csrc/pi_torch.cpp), bound to the loaded library; raises if it was never built."""
    global _native_module
    if _native_module is None:
        if not os.path.exists(EXT_PATH):
            raise RuntimeError(f"{EXT_PATH} is missing: build it with "
                               "`python -m activation_sparse_decode_threshold_b200.build`")
        import importlib.machinery
        import importlib.util
        import torch  # noqa: F401  (its libraries come first)
        loader = importlib.machinery.ExtensionFileLoader("_pi_torch", EXT_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_pi_torch", loader))
        loader.exec_module(module)
        module.init(*(ctypes.cast(getattr(lib(), f), ctypes.c_void_p).value
                      for f in ("pi_int4_matvec", "pi_kv_append", "pi_kv_read", "pi_paged_attention")))
        _native_module = module
    return _native_module


def _bad(where: str, msg: str):
    raise PiError(PI_ERR_INVALID_ARG, where, msg)


def _fail(result, where: str):
    """What a native call returned instead of None: a status, or the text of a refusal."""
    if isinstance(result, str):
        _bad(where, result)
    _check(result, where)


def _stream_arg(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _stream_on(stream, device: int):
    if stream is None:
        import torch
        return torch.cuda.current_stream(device).cuda_stream
    return _stream(stream)


def _handle_desc(h, kind: str, where: str):
    d = _desc.get(h)
    if d is None or d["kind"] != kind:
        _bad(where, f"not a live {kind} handle")
    return d


def pi_int4_create(q, s, device=None, stream=None) -> int:
    """`q`: uint8 [n_rows x n_cols/2] nibbles, `s`: float16 [n_rows x n_cols/32], both contiguous on the device."""
    import torch
    w = "pi_int4_create"
    if not (q.is_cuda and s.is_cuda):
        _bad(w, "q and s must be CUDA tensors")
    device = q.get_device() if device is None else device
    if q.get_device() != device or s.get_device() != device:
        _bad(w, f"q or s is not on cuda:{device}")
    if q.dim() != 2 or q.dtype != torch.uint8 or not q.is_contiguous():
        _bad(w, "q must be contiguous uint8 [n, k/2]")
    n, k = q.shape[0], 2 * q.shape[1]
    if k % 32 or s.dtype != torch.float16 or not s.is_contiguous() or s.shape != (n, k // 32):
        _bad(w, "s must be contiguous float16 [n, k/32]")
    call, h = _native().matvec, ctypes.c_void_p()
    _check(lib().pi_int4_create(n, k, q.data_ptr(), s.data_ptr(), device, _stream_on(stream, device), ctypes.byref(h)), w)
    _desc[h.value] = {"kind": "int4", "shape": (n, k, device), "call": call}
    return h.value


def pi_int4_destroy(m: int):
    if m and _desc.pop(m, None):
        lib().pi_int4_destroy(m)


def pi_int4_matvec(m, x, y, add=None, norm_eps=0.0, stream=None):
    """y [tokens x n_rows] = add + W f(x), x [tokens x n_cols]."""
    d = _handle_desc(m, "int4", "pi_int4_matvec")
    n, k, device = d["shape"]
    got = d["call"](m, n, k, device, x, y, add, norm_eps, stream if stream is None else _stream_arg(stream))
    if got is not None:
        _fail(got, "pi_int4_matvec")


def pi_attn_create(n_heads, n_kv_heads, head_dim, cache_dtype="bf16", page_size=64, layout="hnd", rotary_dim=0,
                   rotary_pairs=False, rope_theta=10000.0, norm_eps=0.0, scale=0.0, softcap=0.0, window=0,
                   device=0) -> int:
    w = "pi_attn_create"
    code = {"i8": DTYPE["i8row"]}.get(cache_dtype, DTYPE.get(cache_dtype))
    if code is None:
        _bad(w, f"unknown cache_dtype {cache_dtype!r}")
    if layout not in KV_LAYOUT:
        _bad(w, f"unknown layout {layout!r}")
    desc = pi_attn_desc(n_heads, n_kv_heads, head_dim, code, page_size, KV_LAYOUT[layout], rotary_dim, int(rotary_pairs),
                        rope_theta, norm_eps, scale, softcap, window, device)
    _native()
    h = ctypes.c_void_p()
    _check(lib().pi_attn_create(ctypes.byref(desc), ctypes.byref(h)), w)
    _desc[h.value] = {"kind": "attention", "device": device, "format": (code, page_size, KV_LAYOUT[layout]),
                      "layer": (h.value, n_heads, n_kv_heads, head_dim, device)}
    return h.value


def pi_attn_destroy(a: int):
    if a and _desc.pop(a, None):
        lib().pi_attn_destroy(a)


def pi_attn_sync(a, stream=None) -> int:
    """Returns the status (does not raise): PI_ERR_DEVICE_CHECK after an index out of range."""
    return lib().pi_attn_sync(a, _stream_on(stream, _handle_desc(a, "attention", "pi_attn_sync")["device"]))


class pi_kv_cache:
    """The tensors of one layer's cache: k and v [pages, kv heads, page size, row] ("hnd") or [pages, page size, kv
    heads, row] ("nhd") with row = head_dim values (float16, bfloat16, int8) or head_dim/2 bytes (int4g32: uint8);
    scales without the row (float32) for int8, with head_dim/32 float16 for int4g32.  The four tensors are the cache's for
    good; their memory and shapes are taken, and checked against the handle's format, at each call."""

    __slots__ = ("_tensors", "_last")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self._tensors, self._last = (k, v, k_scale, v_scale), (None, None)

    k, v, k_scale, v_scale = (property(lambda self, i=i: self._tensors[i]) for i in range(4))


def _cache_arg(cache, d):
    """The tuple that the native part takes: the format that the handle expects, and the tensors."""
    of, arg = cache._last
    if of is not d:
        arg = (*d["format"], *cache._tensors)
        cache._last = d, arg   # (both at once: threads may use a cache with handles of their own)
    return arg


def pi_kv_append(a, cache, table, pos, q, k, v, q_out, seq=None, q_norm=None, k_norm=None, stream=None):
    """q, q_out [tokens, heads, dim], k and v [tokens, kv heads, dim]; `pos` (and `seq`) int32 [tokens]."""
    d = _handle_desc(a, "attention", "pi_kv_append")
    got = _native_module.append(d["layer"], _cache_arg(cache, d), table, pos, q, k, v, q_out, seq, q_norm, k_norm,
                                stream if stream is None else _stream_arg(stream))
    if got is not None:
        _fail(got, "pi_kv_append")


def pi_kv_read(a, cache, table, pos, k_out, v_out, seq=None, stream=None):
    """k_out and v_out: contiguous [tokens, kv heads, dim] of one type."""
    d = _handle_desc(a, "attention", "pi_kv_read")
    got = _native_module.read(d["layer"], _cache_arg(cache, d), table, pos, k_out, v_out, seq,
                              stream if stream is None else _stream_arg(stream))
    if got is not None:
        _fail(got, "pi_kv_read")


def pi_paged_attention(a, cache, table, lens, q, out, lse=None, stream=None):
    """q and out [sequences, heads, dim]; `lens` int32 [sequences]; `lse` float32 [sequences, heads] or None."""
    d = _handle_desc(a, "attention", "pi_paged_attention")
    got = _native_module.attend(d["layer"], _cache_arg(cache, d), table, lens, q, out, lse,
                                stream if stream is None else _stream_arg(stream))
    if got is not None:
        _fail(got, "pi_paged_attention")
