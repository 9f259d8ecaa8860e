"""The attention half of a decode layer at the limits of its numbers: the largest
values, few rounded steps, long exact sums.  Definitions and roundings: attn_ref.py."""
import math

import pytest
import torch

import attn_ref as R
from activation_sparse_decode_threshold_b200 import binding as B
from test_gpu_attention import attend, cache_of, check, gen, layer, made, matrix, refused  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,tokens", [(40, 96, 1), (33, 416, 3), (70, 8192, 13)])
def test_matvec_largest_numbers(made, dt, n, k, tokens):
    """x up to the type's largest number: as long as the result is finite, so is every sum on the way to it."""
    g = gen(n + tokens)
    q, _ = R.encode_int4(torch.randn(n, k, generator=g))
    s = torch.full((n, k // 32), 2.0 ** -14, dtype=torch.float16)      # |y| <= 8 K 2^-14 max |x| / (random signs)
    top = torch.finfo(R.DT[dt]).max
    x = ((0.5 + 0.5 * torch.rand(tokens, k, generator=g)) * torch.where(torch.rand(tokens, k, generator=g) < 0.5, -1.0, 1.0)).double()
    x = (x * top).to(R.DT[dt]).clamp(-top, top)
    x[0] = x[0].abs()                                                  # (one token without the signs' help)
    x[0, ::2] = top
    y = torch.zeros(tokens, n, device="cuda")
    B.pi_int4_matvec(matrix(made, q, s), x.cuda(), y)
    want, bound = R.matvec(q, s, x, torch.float32)
    assert want.abs().max() < 0.9 * top
    check(y, want, bound)
