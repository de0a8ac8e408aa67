"""Prompt attention over many units of work, which the CTAs take whole, one after the other, off a list: every row of
batches of many items, heads and sizes, and every kind of pool, against 64-bit torch."""

import random

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import attend, check, ints, starts_of
from test_gpu_prompt import check_prefill, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _workspace(pool, seqs, hq, rows, most):
    return torch.zeros(pkv.prefill_workspace_bytes(pool, seqs, hq, rows, most), dtype=torch.uint8, device="cuda")


def _took_whole_items(ws):
    """The plan's second word tells the two forms of its list apart: 1 is the line that is cut."""
    return ws[:8].view(torch.int32)[1].item() == 0


def _batch(seed, seqs, hi):
    """Sequences of up to hi new tokens, single tokens and empty ones among them, and the tokens before them."""
    rng = random.Random(seed)
    new = [rng.choice([0, 1, 1, rng.randint(2, hi), rng.randint(2, hi), rng.randint(hi // 2, hi)]) for _ in range(seqs)]
    return new, [rng.choice([0, 0, rng.randint(1, 40), rng.randint(100, 400)]) for _ in range(seqs)]


# heads, and sequences enough for the list on 152 SMs: some 2000 to 4000 units of work
SHAPES = [(32, 32, 128, 64, 700), (32, 8, 128, 130, 420), (28, 4, 64, 330, 200), (32, 32, 64, 96, 500), (71, 1, 64, 380, 60),
          (160, 1, 128, 420, 30)]


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("hq,hkv,d,seqs,hi", SHAPES)
def test_prefill(hq, hkv, d, seqs, hi, window, kv):
    new, before = _batch(hq + d + window, seqs, hi)
    lens = [a + b for a, b in zip(new, before)]
    gen = torch.Generator(device="cuda").manual_seed(seqs)
    pool, tables = make_cache(gen, lens, hkv, d, kv)
    n = sum(new)
    q = torch.randn(n + 3, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    ws = _workspace(pool, seqs, hq, n + 3, max(lens))
    args = (q, tables, ints(lens), starts_of(new), d ** -0.5, max(lens))
    pool.prefill(*args, window=window, out=out, workspace=ws)
    assert pool.device_error() == 0 and _took_whole_items(ws)
    check_prefill(pool, tables, q, out, new, lens, d ** -0.5, window, (hq, hkv, d, kv, window))
    assert (out[n:] == 7.0).all()
    for _ in range(3):
        assert torch.equal(pool.prefill(*args, window=window)[:n], out[:n])
    pool.close()


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 150), (False, 0)])
@pytest.mark.parametrize("hq,hkv,d,seqs,hi", SHAPES)
def test_prompts(hq, hkv, d, seqs, hi, causal, window):
    new, before = _batch(hq + d + causal, seqs, hi)
    before = [b if i % 3 else -min(new[i], 9) for i, b in enumerate(before)]  # fewer keys than queries too
    keys = [a + b for a, b in zip(new, before)]
    gen = torch.Generator(device="cuda").manual_seed(seqs + 1)
    pool = pkv.PagedKVPool(2, hkv, d, "bf16")
    n, m = sum(new), sum(keys)
    q = torch.randn(n + 2, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
    x = torch.randn(m + 2, 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
    k, v = x[:, :hkv], x[:, hkv:]
    k[m:], v[m:] = float("nan"), float("inf")
    out = torch.full_like(q, 7.0)
    ws = _workspace(pool, seqs, hq, n + 2, m + 2)
    pool.prompt_attention(q, k, v, starts_of(new), d ** -0.5, key_starts=starts_of(keys), causal=causal, window=window, out=out,
                          workspace=ws)
    assert pool.device_error() == 0 and _took_whole_items(ws)
    at = key = 0
    for b, (nb, t) in enumerate(zip(new, keys)):
        ref = attend(q[at:at + nb].double(), k[key:key + t].double(), v[key:key + t].double(), d ** -0.5, window, causal)
        check(out[at:at + nb], *ref, t, (b, nb, t))
        at, key = at + nb, key + t
    assert (out[n:] == 7.0).all()
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_every_sequence_of_many_small_ones(kv):
    new = [1, 40, 130, 2, 0, 70] * 40
    lens = [1 + n + (i * 37) % 300 for i, n in enumerate(new)]
    gen = torch.Generator(device="cuda").manual_seed(9)
    pool, tables = make_cache(gen, lens, 8, 64, kv)
    q = torch.randn(sum(new), 32, 64, generator=gen, device="cuda").to(torch.bfloat16)
    ws = _workspace(pool, len(new), 32, len(q), max(lens))
    out = pool.prefill(q, tables, ints(lens), starts_of(new), 0.125, max(lens), workspace=ws)
    assert pool.device_error() == 0 and _took_whole_items(ws)
    check_prefill(pool, tables, q, out, new, lens, 0.125, 0, kv)
    pool.close()


@pytest.mark.parametrize("seqs", [1024, 1025, 3000])
def test_every_sequence_of_thousands(seqs):
    """Of up to 1024 sequences the plan holds what it needs in shared memory, of more it does not."""
    new = [(i * 7) % 4 for i in range(seqs)]
    lens = [n + (i * 13) % 40 for i, n in enumerate(new)]
    gen = torch.Generator(device="cuda").manual_seed(11)
    pool, tables = make_cache(gen, lens, 2, 64, "bf16")
    q = torch.randn(sum(new), 4, 64, generator=gen, device="cuda").to(torch.bfloat16)
    ws = _workspace(pool, seqs, 4, len(q), 80)
    out = pool.prefill(q, tables, ints(lens), starts_of(new), 0.125, 80, workspace=ws)
    assert pool.device_error() == 0 and _took_whole_items(ws)
    check_prefill(pool, tables, q, out, new, lens, 0.125, 0, seqs)
    pool.close()
