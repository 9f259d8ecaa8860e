"""Refusals of the attention half of a decode layer that need no GPU."""
import ctypes

import pytest
import torch

from activation_sparse_decode_threshold_b200 import binding as B


def _desc(**kw):
    base = dict(n_heads=32, n_kv_heads=8, head_dim=128, cache_dtype=2, page_size=64, layout=0, rotary_dim=128,
                rotary_pairs=0, rope_theta=10000.0, norm_eps=1e-6, scale=0.0, softcap=0.0, window=0, device=0)
    base.update(kw)
    return B.pi_attn_desc(**base)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad, status", [
    (dict(n_kv_heads=0), B.PI_ERR_INVALID_ARG),
    (dict(n_kv_heads=5), B.PI_ERR_INVALID_ARG),
    (dict(n_heads=2048), B.PI_ERR_INVALID_ARG),
    (dict(n_heads=0), B.PI_ERR_INVALID_ARG),
    (dict(head_dim=96), B.PI_ERR_UNSUPPORTED),
    (dict(head_dim=256), B.PI_ERR_UNSUPPORTED),
    (dict(cache_dtype=0), B.PI_ERR_UNSUPPORTED),
    (dict(cache_dtype=9), B.PI_ERR_UNSUPPORTED),
    (dict(page_size=4), B.PI_ERR_UNSUPPORTED),
    (dict(page_size=24), B.PI_ERR_UNSUPPORTED),
    (dict(page_size=512), B.PI_ERR_UNSUPPORTED),
    (dict(layout=2), B.PI_ERR_INVALID_ARG),
    (dict(rotary_dim=130), B.PI_ERR_INVALID_ARG),
    (dict(rotary_dim=3), B.PI_ERR_INVALID_ARG),
    (dict(rotary_dim=-2), B.PI_ERR_INVALID_ARG),
    (dict(rotary_pairs=2), B.PI_ERR_INVALID_ARG),
    (dict(rope_theta=0.0), B.PI_ERR_INVALID_ARG),
    (dict(rope_theta=INF), B.PI_ERR_INVALID_ARG),
    (dict(norm_eps=-1.0), B.PI_ERR_INVALID_ARG),
    (dict(norm_eps=NAN), B.PI_ERR_INVALID_ARG),
    (dict(scale=INF), B.PI_ERR_INVALID_ARG),
    (dict(softcap=-1.0), B.PI_ERR_INVALID_ARG),
    (dict(softcap=NAN), B.PI_ERR_INVALID_ARG),
    (dict(window=-1), B.PI_ERR_INVALID_ARG),
])
def test_attention_descriptors_are_checked_on_the_host(bad, status):
    h = ctypes.c_void_p()
    assert B.lib().pi_attn_create(ctypes.byref(_desc(**bad)), ctypes.byref(h)) == status, B.pi_last_error()
    assert h.value is None and B.pi_last_error()


@pytest.mark.parametrize("n, k, q, s", [(0, 64, 16, 16), (2 ** 20 + 1, 64, 16, 16), (8, 0, 16, 16), (8, 48, 16, 16),
                                        (8, 2 ** 17 + 32, 16, 16), (8, 64, None, 16), (8, 64, 16, None), (8, 64, 24, 16),
                                        (8, 64, 16, 17)])
def test_int4_matrices_are_checked_on_the_host(n, k, q, s):
    h = ctypes.c_void_p()
    assert B.lib().pi_int4_create(n, k, q, s, 0, None, ctypes.byref(h)) == B.PI_ERR_INVALID_ARG
    assert h.value is None and B.pi_last_error()


def test_null_arguments_are_refused():
    L = B.lib()
    assert L.pi_int4_create(8, 64, 16, 16, 0, None, None) == B.PI_ERR_INVALID_ARG
    assert L.pi_int4_matvec(None, 1, 0, None, 0, None, 0, None, 0, 0.0, None) == B.PI_ERR_INVALID_ARG
    assert L.pi_attn_create(None, None) == B.PI_ERR_INVALID_ARG
    assert L.pi_attn_sync(None, None) == B.PI_ERR_INVALID_ARG
    assert L.pi_kv_append(None, None, None, 1, None, None, 0, None, 0, None, 0, None, 0, None, None, None, 0,
                          None) == B.PI_ERR_INVALID_ARG
    assert L.pi_kv_read(None, None, None, 1, None, None, 0, None, None, None) == B.PI_ERR_INVALID_ARG
    assert L.pi_paged_attention(None, None, None, None, 0, None, 0, None, 0, None, None) == B.PI_ERR_INVALID_ARG
    L.pi_int4_destroy(None)
    L.pi_attn_destroy(None)


def test_binding_refuses_tensors_of_the_host():
    q = torch.zeros(8, 32, dtype=torch.uint8)
    with pytest.raises(B.PiError) as e:
        B.pi_int4_create(q, torch.zeros(8, 2, dtype=torch.float16))
    assert e.value.status == B.PI_ERR_INVALID_ARG
    with pytest.raises(B.PiError):
        B.pi_int4_matvec(1234, q, q)
    with pytest.raises(B.PiError):
        B.pi_attn_create(8, 2, 64, cache_dtype="f64")
    with pytest.raises(B.PiError):
        B.pi_attn_create(8, 2, 64, layout="dhn")
