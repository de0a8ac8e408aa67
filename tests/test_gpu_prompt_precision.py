"""Prompt attention within the bounds of the roundings that it is documented to have, each by itself (prompt_bounds.py):
few tokens to a query, whose values nearly cancel or all have one sign, and whole contexts."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_bounds import tight
from prompt_reference import attend, cached, ints, starts_of
from test_gpu_prompt import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _within(got, ref, tokens, codes, what):
    bound = tight(*ref, tokens, got.shape[-1], codes)
    over = ((got.double() - ref[0]).abs() / bound).nan_to_num(1e9).max().item()
    assert over <= 1, (what, over)


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (4, 4, 128)])
@pytest.mark.parametrize("window", [2, 3, 8, 40, 0])
@pytest.mark.parametrize("signs", ["both", "one"])
def test_prefill(kv, hq, hkv, d, window, signs):
    gen = torch.Generator(device="cuda").manual_seed(window + d)
    new, lens = [300, 20, 1, 1], [300, 900, 5, 2000]
    pool, tables = make_cache(gen, lens, hkv, d, kv)
    if signs == "one":
        pool.v_cache.copy_(pool.v_cache.abs() if kv == "bf16" else pool.v_cache & 127 if kv == "fp8" else pool.v_cache.clamp(min=0))
    q = torch.randn(sum(new), hq, d, generator=gen, device="cuda").to(torch.bfloat16)
    out = pool.prefill(q, tables, ints(lens), starts_of(new), d ** -0.5, max(lens), window=window)
    at = 0
    for b, (n, t) in enumerate(zip(new, lens)):
        k, v, _ = cached(pool, tables[b], t)
        ref = attend(q[at:at + n].double(), k, v, d ** -0.5, window)
        _within(out[at:at + n], ref, min(t, window or t), kv != "bf16", (kv, d, window, b))
        at += n
    pool.close()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts(d, causal):
    gen = torch.Generator(device="cuda").manual_seed(d)
    new = [2, 3, 8, 300, 1000]
    x = torch.randn(sum(new), 12, d, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    pool = pkv.PagedKVPool(2, 2, d, "bf16")
    out = pool.prompt_attention(q, k, v, starts_of(new), d ** -0.5, causal=causal)
    at = 0
    for n in new:
        rows = slice(at, at + n)
        _within(out[rows], attend(q[rows].double(), k[rows].double(), v[rows].double(), d ** -0.5, causal=causal), n, False, n)
        at += n
    pool.close()
