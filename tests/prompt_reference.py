"""Attention of packed queries in 64-bit torch, and how far the kernels may be from it."""

from __future__ import annotations

import torch

BLOCK = 16


def attend(q, k, v, scale, window=0, causal=True, missing=None):
    """q [n, Hq, d], k and v [T, Hkv, d] in 64 bits -> (out [n, Hq, d], W, A, M): W = sum of weight |v| for
    each output, A = the largest sum |q k| scale of a logit for each row, M [.., 2] = the row's largest weight |v| of a
    token's largest value, and the largest |v| it sees.  ``missing``: tokens [T] that are
    not there."""
    n, hq, d = q.shape
    t, hkv = k.shape[:2]
    g = hq // hkv
    rows = q.view(n, hkv, g, d)
    x = torch.einsum("nhgd,thd->hgnt", rows, k) * scale
    size = torch.einsum("nhgd,thd->hgnt", rows.abs(), k.abs()) * abs(scale)
    pos = torch.arange(t - n, t, device=q.device)[:, None]
    col = torch.arange(t, device=q.device)
    seen = col <= pos if causal else torch.ones(n, t, dtype=torch.bool, device=q.device)
    if window:
        seen = seen & (col > pos - window)
    if missing is not None:
        seen = seen & ~missing
    x = x.masked_fill(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True) if t else torch.zeros(hkv, g, n, 1, device=q.device, dtype=q.dtype)
    w = torch.exp(x - torch.where(top.isinf(), 0.0, top)).masked_fill(~seen, 0.0)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0)
    vz = torch.where(seen.any(0)[:, None, None], v, 0.0)  # what nobody sees may hold anything
    a = size.masked_fill(~seen, 0.0).amax(-1) if t else torch.zeros(hkv, g, n, device=q.device, dtype=q.dtype)

    def back(y):
        return y.permute(2, 0, 1, 3).reshape(n, hq, y.shape[-1])

    out = back(torch.einsum("hgnt,thd->hgnd", w, vz))
    size_v = vz.abs().amax(-1).transpose(0, 1)[:, None, None]  # [Hkv, 1, 1, t]
    peak = torch.stack([w * size_v, seen * size_v.expand_as(w)], -1).amax(-2) if t else torch.zeros(hkv, g, n, 2, device=q.device)
    return out, back(torch.einsum("hgnt,thd->hgnd", w, vz.abs())), back(a[..., None]), back(peak)


def tolerance(out, weight, size, peak, tokens, d, codes):
    """Largest error of an output, from the arithmetic:

    - a weight enters the product over V as bf16 (2^-8 of it; over codes as fp16, 2^-11), the softmax sum may or may not
      use the rounded ones (2^-8 of the output), and the output is rounded to bf16 (2^-8 of it);
    - a logit is a sum of d products in fp32, d + 2 steps of at most 2^-23 of sum |q k|, then scaled and shifted: it moves
      by at most 2^-23 (d + 8) A, and the weights, numerator and sum, by twice that;
    - exponentials, the sums over the tokens and the rescaling: 2^-22 and `tokens` steps of 2^-23 of W;
    - over codes a weight times its token's scale is held relative to the row's largest such, which is at least 2^-1:
      below 2^-14 fp16's steps are 2^-24, off by half a step, 2^-25, so 2^-24 of the largest, for each token; a
      token's largest value is its scale times 127 or 448, so in values it is 2^-24 of the row's largest weight |v|;
    - exponentials below 2^-126 are 0, 2^-117 of the largest at most: the maximum may stand 2^8 too low."""
    move = 2.0 ** -23 * (d + 8) * size
    tol = (2.0 ** -8 * (weight + 2 * out.abs()) * (1 + 2.0 ** -7)
           + (torch.expm1(2 * move) + 2.0 ** -20 + tokens * 2.0 ** -23) * (weight + out.abs()) + 1e-30)
    if codes:
        tol = tol + 2.0 ** -24 * tokens * peak[..., :1]
    return tol + 2.0 ** -117 * tokens * peak[..., 1:]


def check(got, ref, weight, size, peak, tokens, what, codes=False):
    tol = tolerance(ref, weight, size, peak, tokens, ref.shape[-1], codes)
    bad = ~((got.double() - ref).abs() <= tol)  # a NaN is bad
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           ((got.double() - ref).abs() / tol).nan_to_num(1e9).max().item())


def cached(pool, table, t):
    """(K, V, missing) of a sequence's first t tokens in 64 bits: [t, Hkv, d]."""
    blocks = table[:(t + BLOCK - 1) // BLOCK].long()
    there = (blocks >= 0) & (blocks < pool.num_blocks)
    at = torch.where(there, blocks, 0)
    out = []
    for cache, scale in ((pool.k_cache, pool.k_scale), (pool.v_cache, pool.v_scale)):
        x = cache[at]
        x = (x.view(torch.float8_e4m3fn).float() if pool.dtype == "fp8" else x).double()
        if pool.dtype != "bf16":
            x = x * scale[at].double()[..., None]
        out.append(x.transpose(1, 2).flatten(0, 1)[:t])
    return out[0], out[1], ~there.repeat_interleave(BLOCK)[:t]


def starts_of(sizes):
    s = [0]
    for n in sizes:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")
