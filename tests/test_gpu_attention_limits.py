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


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,tokens", [(40, 96, 1), (33, 416, 7), (70, 8192, 13), (24, 8192, 32)])
def test_matvec_norm_of_large_and_small_numbers(made, dt, n, k, tokens):
    """Tokens whose squares leave fp32's range (above 1.8e19), beside ordinary ones, zeros and small ones."""
    g = gen(n + tokens)
    q, s = R.encode_int4(torch.randn(n, k, generator=g) * 0.05)
    sizes = torch.tensor([1e20, 1.0, 1e30, 0.0, 1e36, 1e19, 1e-20])[torch.arange(tokens) % 7]
    x = (torch.randn(tokens, k, generator=g) * sizes[:, None]).to(R.DT[dt])
    if tokens > 1:
        x[1, 5] = 1e22                                                 # one large element among ordinary ones
    y = torch.zeros(tokens, n, device="cuda")
    B.pi_int4_matvec(matrix(made, q, s), x.cuda(), y, norm_eps=1e-6)
    want, bound = R.matvec(q, s, x, torch.float32, eps=1e-6)
    check(y, want, bound)
    # without a norm the same numbers stay apart too: nothing of one token gets into another
    alone = torch.zeros(1, n, device="cuda")
    for t in (0, tokens - 1):
        B.pi_int4_matvec(matrix(made, q, s), x[t:t + 1].cuda(), alone, norm_eps=1e-6)
        want, bound = R.matvec(q, s, x[t:t + 1], torch.float32, eps=1e-6)
        check(alone, want, bound)
