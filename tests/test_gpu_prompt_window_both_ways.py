"""prompt_attention without the causal limit and with a window: query i of n sees every key t of its sequence's T
with t > T - n + i - window, those behind it included."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import attend, check, ints, starts_of
from test_gpu_prompt import run_prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("window", [1, 2, 17, 127, 128, 129, 300, 900, 5000])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (14, 2, 64), (4, 4, 128), (71, 1, 64)])
def test_windows(window, hq, hkv, d):
    """More keys than queries, as many, fewer, one, none."""
    run_prompt(window + d, [5, 200, 40, 0, 7, 300, 1], [100, 20, 0, 50, 7, 1111, 1], hq, hkv, d, causal=False, window=window)


@pytest.mark.parametrize("window", [1, 100, 4000, 16500, 20000])
@pytest.mark.parametrize("d", [64, 128])
def test_long_keys_are_cut_and_joined(window, d):
    run_prompt(window, [20, 1, 0, 300], [9000, 17000, 30, 17000], 4, 2, d, causal=False, window=window)


@pytest.mark.parametrize("window", [0, 1, 130, 700])
def test_the_queries_rows_as_keys(window):
    """Starts of the keys that are the queries' own."""
    run_prompt(window, [300, 0, 1, 129, 700], [300, 0, 1, 129, 700], 8, 2, 128, causal=False, window=window)


def test_keys_that_nobody_sees_may_hold_anything():
    gen = torch.Generator(device="cuda").manual_seed(4)
    new, keys, w, d = [30, 7], [500, 260], 45, 128
    q = torch.randn(sum(new), 8, d, generator=gen, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(sum(keys), 2, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    k64, v64, at = k.double(), v.double(), 0
    for n, t in zip(new, keys):
        first = t - n - w + 1  # the first key that any query sees
        k[at:at + first] = float("nan")
        v[at:at + first] = float("inf")
        at += t
    pool = pkv.PagedKVPool(2, 2, d, "bf16")
    out = pool.prompt_attention(q, k, v, starts_of(new), 0.1, key_starts=starts_of(keys), causal=False, window=w)
    at = key = 0
    for n, t in zip(new, keys):
        ref = attend(q[at:at + n].double(), k64[key:key + t], v64[key:key + t], 0.1, w, False)
        check(out[at:at + n], *ref, t, (n, t))
        at, key = at + n, key + t
    assert pool.device_error() == 0
    pool.close()


def test_refused_without_starts_of_the_keys():
    pool = pkv.PagedKVPool(2, 2, 64, "bf16")
    q, k = (torch.zeros(6, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    before = pkv.launch_count()
    with pytest.raises(pkv.PagedKVError):
        pool.prompt_attention(q, k, k, ints([0, 3, 6]), 0.1, causal=False, window=5)
    with pytest.raises(pkv.PagedKVError):
        pool.prompt_attention(q, k, k, ints([0, 3, 6]), 0.1, key_starts=ints([0, 3, 6]), causal=False, window=-1)
    assert pkv.launch_count() == before
    pool.close()
