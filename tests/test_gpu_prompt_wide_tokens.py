"""The prompt operators with as many heads as they take: a token's queries, keys or values are at most 2^27 - 1 values,
so that a head's place within a token or a block is a 32-bit number."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import attend, check, ints

pytestmark = pytest.mark.gpu

D = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("heads", [2 ** 21, 2 ** 21 + 8])
def test_wider_tokens_are_refused(heads):
    pool = pkv.PagedKVPool(1, heads, D, "int8")
    x = torch.zeros(1, heads, D, dtype=torch.bfloat16, device="cuda")
    table, one, starts = ints([[0]]), ints([1]), ints([0, 1])
    before = pkv.launch_count()
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for call in (lambda: pool.prefill(x, table, one, starts, 0.1, 16, workspace=ws),
                 lambda: pool.prompt_attention(x, x, x, starts, 0.1, workspace=ws),
                 lambda: pool.gather_cache(table, starts, 1, k=x, v=x.clone()),
                 lambda: pkv.prefill_workspace_bytes(pool, 1, heads, 1, 16)):
        with pytest.raises(pkv.PagedKVError, match="unsupported"):
            call()
    assert pkv.launch_count() == before
    pool.close()


def test_queries_wider_than_the_keys_are_refused():
    pool = pkv.PagedKVPool(1, 8, D, "bf16", fill=0)
    x = torch.zeros(1, 2 ** 21, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PagedKVError, match="unsupported"):
        pool.prefill(x, ints([[0]]), ints([1]), ints([0, 1]), 0.1, 16, workspace=x)
    with pytest.raises(pkv.PagedKVError, match="unsupported"):
        pool.prompt_attention(x, x[:, :8], x[:, :8], ints([0, 1]), 0.1, workspace=x)
    pool.close()


def test_the_widest_tokens():
    heads, t = 2 ** 21 - 8, 11
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool = pkv.PagedKVPool(1, heads, D, "int8")
    pool.k_cache.random_(-127, 128, generator=gen)
    pool.v_cache.random_(-127, 128, generator=gen)
    pool.k_scale.uniform_(0.005, 0.02, generator=gen)
    pool.v_scale.uniform_(0.005, 0.02, generator=gen)
    q = torch.randn(2, heads, D, generator=gen, device="cuda").to(torch.bfloat16)
    out = pool.prefill(q, ints([[0]]), ints([t]), ints([0, 2]), 0.125, 16)
    k, v = pool.gather_cache(ints([[0]]), ints([0, 2]), 2)
    packed = pool.prompt_attention(q, k, v, ints([0, 2]), 0.125)
    assert pool.device_error() == 0
    for lo in (0, heads // 2, heads - 4096):
        part = slice(lo, lo + 4096)
        exact = [(c[0, part].double() * s[0, part].double()[..., None])[:, :t].transpose(0, 1)
                 for c, s in ((pool.k_cache, pool.k_scale), (pool.v_cache, pool.v_scale))]
        check(out[:, part], *attend(q[:, part].double(), *exact, 0.125), t, lo, True)
        for got, ref in zip((k, v), exact):
            assert ((got[:, part].double() - ref[:2]).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref[:2].abs()).all()
        check(packed[:, part], *attend(q[:, part].double(), k[:, part].double(), v[:, part].double(), 0.125), 2, lo)
    pool.close()
