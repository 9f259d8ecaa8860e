"""The binding's native part on the host: what it answers to arguments that are not
what the entry points take (nothing is launched)."""
import torch

from activation_sparse_decode_threshold_b200 import binding as B

LAYER = (0, 4, 2, 64, 0)


def test_tensors_of_the_host_are_refused_by_name():
    n, t = B._native(), torch.zeros(2, 64)
    i = torch.zeros(2, dtype=torch.int32)
    assert n.matvec(0, 8, 64, 0, t, t, None, 0.0, 0) == "x is not on cuda:0"
    assert n.append(LAYER, 0, i, i, t, t, t, t, None, None, None, 0) == "table is not on cuda:0"
    assert n.read(LAYER, 0, i, i, t, t, None, 0) == "table is not on cuda:0"
    assert n.attend(LAYER, 0, i, i, t, t, None, 0) == "table is not on cuda:0"


def test_what_is_no_tensor_is_refused():
    n = B._native()
    for x in (None, 1.5, "x", [1, 2]):
        assert n.matvec(0, 8, 64, 0, x, x, None, 0.0, 0) == "x must be a tensor"
        assert n.attend(LAYER, 0, x, x, x, x, None, 0) == "table must be a tensor"


def test_layers_and_argument_counts_are_checked():
    n = B._native()
    assert n.attend((1, 2), 0, None, None, None, None, None, 0) == "not a layer"
    assert "arguments instead of 9" in n.matvec(0, 8)
    assert "arguments instead of 12" in n.append()
    for bad in (("a", 4, 2, 64, 0), (2 ** 80, 4, 2, 64, 0)):
        try:
            n.attend(bad, 0, None, None, None, None, None, 0)
        except (TypeError, OverflowError):
            continue
        raise AssertionError("no exception")


def test_a_refusal_becomes_the_binding_s_error():
    for got, status in (("text of a refusal", B.PI_ERR_INVALID_ARG), (B.PI_ERR_CUDA, B.PI_ERR_CUDA)):
        try:
            B._fail(got, "pi_kv_read")
        except B.PiError as e:
            assert e.status == status and "pi_kv_read" in str(e)
            continue
        raise AssertionError("no error")
