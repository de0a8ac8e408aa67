"""The bounds on prompt attention's precision tell its roundings apart: outputs with the roundings that the kernels
have lie within them, outputs with a rounding more do not."""

import pytest
import torch

from prompt_bounds import tight
from prompt_reference import attend


def _problem(codes, d=64, n=40, t=43):
    """Few tokens to a query (window 3), whose values nearly cancel."""
    gen = torch.Generator().manual_seed(1 + codes)
    q = torch.randn(n, 4, d, generator=gen).to(torch.bfloat16).double()
    k = torch.randn(t, 2, d, generator=gen).to(torch.bfloat16).double()
    v = torch.randn(t, 2, d, generator=gen)
    v = (32 * v).round().clamp(-127, 127).double() * 0.03 if codes else v.to(torch.bfloat16).double()
    return q, k, v


def _emulated(q, k, v, scale, window, weights, sums):
    """Attention with the weights of the product over V rounded to one type and those of the sum to another."""
    n, hq, d = q.shape
    t, hkv = k.shape[:2]
    x = torch.einsum("nhgd,thd->hgnt", q.view(n, hkv, hq // hkv, d), k) * scale
    away = torch.arange(t - n, t)[:, None] - torch.arange(t)
    x = x.masked_fill((away < 0) | (away >= window), float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))

    def rounded(y, to):
        return y if to is None else y.to(to).double()

    o = torch.einsum("hgnt,thd->nhgd", rounded(p, weights) / rounded(p, sums).sum(-1, keepdim=True), v)
    return o.reshape(n, hq, d).to(torch.bfloat16).double()


@pytest.mark.parametrize("codes", [False, True])
def test_the_kernels_roundings_lie_within(codes):
    q, k, v = _problem(codes)
    ref = attend(q, k, v, 0.125, 3)
    got = _emulated(q, k, v, 0.125, 3, torch.float16 if codes else torch.bfloat16, None)
    assert ((got - ref[0]).abs() <= tight(*ref, 3, 64, codes)).all()


def test_over_codes_weights_of_bf16_do_not():
    q, k, v = _problem(True)
    ref = attend(q, k, v, 0.125, 3)
    got = _emulated(q, k, v, 0.125, 3, torch.bfloat16, None)
    assert ((got - ref[0]).abs() > tight(*ref, 3, 64, True)).any()


def test_over_bf16_weights_of_fewer_bits_do_not():
    q, k, v = _problem(False)
    ref = attend(q, k, v, 0.125, 3)
    got = _emulated(q, k, v, 0.125, 3, torch.float8_e4m3fn, None)
    assert ((got - ref[0]).abs() > tight(*ref, 3, 64, False)).any()


def test_over_codes_a_sum_of_weights_of_bf16_does_not():
    """Values of one sign, so that the sum of weight |v| is the output itself and leaves room for one rounding of it."""
    q, k, v = _problem(True)
    v = v.abs()
    ref = attend(q, k, v, 0.125, 3)
    right, wrong = (_emulated(q, k, v, 0.125, 3, torch.float16, to) for to in (None, torch.bfloat16))
    bound = tight(*ref, 3, 64, True)
    assert ((right - ref[0]).abs() <= bound).all() and ((wrong - ref[0]).abs() > bound).any()
