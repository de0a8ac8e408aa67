"""How far prompt attention may be from 64-bit torch, each of its roundings by itself.

Over bf16 a weight enters the product over V as bf16, over codes as fp16; the softmax sum is over unrounded weights."""

from __future__ import annotations

import torch


def tight(out, weight, size, peak, tokens, d, codes):
    """Largest error of an output; the arguments are ``prompt_reference.attend``'s.

    - A weight in the product over V is off by half a step: 2^-8 of it as bf16, 2^-11 as fp16, and with it the sum of
      weight |v|.  The sum of the weights is over unrounded ones.
    - The output is rounded to bf16: 2^-8 of it, and of the error that it has by then (the factor 1 + 2^-7).
    - A logit is a sum of d products in fp32, d + 8 steps of 2^-23 of sum |q k| with scaling and shift, and moves numerator
      and sum by twice that; exponentials, rescaling and division 2^-20, the sums 2^-23 a token, in both.
    - Over codes a weight below 2^-14 is off by 2^-25 at most, where the row's largest weight times scale is at least 2^-1 in
      the same units: 2^-24 of the row's largest weight |v| for each token.
    - Exponentials below 2^-126 are 0, with a maximum that may stand 2^8 too low: 2^-117 of the largest |v| a token."""
    move = 2.0 ** -23 * (d + 8) * size
    tol = (((2.0 ** -11 if codes else 2.0 ** -8) * weight + 2.0 ** -8 * out.abs()) * (1 + 2.0 ** -7)
           + (torch.expm1(2 * move) + 2.0 ** -20 + tokens * 2.0 ** -23) * (weight + out.abs()) + 1e-30)
    if codes:
        tol = tol + 2.0 ** -24 * tokens * peak[..., :1]
    return tol + 2.0 ** -117 * tokens * peak[..., 1:]
