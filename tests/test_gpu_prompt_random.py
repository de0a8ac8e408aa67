"""paged_attention_prefill and prompt_attention over batches drawn at random: sequences without queries, single
tokens, chunks of any size and long contexts side by side, against 64-bit torch; the same call again gives the
same bits."""

import random

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import ints, starts_of
from test_gpu_prompt import check_prefill, make_cache, run_prompt

pytestmark = pytest.mark.gpu

HEADS = [(8, 2, 64), (4, 4, 128), (28, 4, 128), (16, 1, 64), (5, 1, 128), (32, 32, 64)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _batch(rng):
    seqs = rng.choice([1, 2, 5, 20, 60])
    new, before = [], []
    for _ in range(seqs):
        kind = rng.choice(["one", "one", "none", "few", "chunk", "long"])
        n = {"one": 1, "none": 0, "few": rng.randint(2, 40), "chunk": rng.randint(60, 400), "long": rng.randint(1, 30)}[kind]
        t = rng.randint(3000, 9000) if kind == "long" and seqs < 20 else rng.choice([0, rng.randint(0, 600)])
        new.append(n)
        before.append(t)
    return new, before


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("seed", range(12))
def test_prefill_batches(seed, kv):
    rng = random.Random(seed * 3 + len(kv))
    new, before = _batch(rng)
    hq, hkv, d = rng.choice(HEADS)
    window = rng.choice([0, 0, 0, rng.randint(1, 700)])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = [a + b for a, b in zip(new, before)]
    pool, tables = make_cache(gen, lens, hkv, d, kv)
    q = (1.5 * torch.randn(sum(new) + 1, hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
    args = (q, tables, ints(lens), starts_of(new), d ** -0.5, max(lens + [1]))
    out = pool.prefill(*args, window=window)
    torch.cuda.synchronize()
    assert pool.device_error() == 0
    check_prefill(pool, tables, q, out, new, lens, d ** -0.5, window, (seed, kv, new, before, hq, hkv, d, window))
    n = sum(new)
    for _ in range(3):
        assert torch.equal(pool.prefill(*args, window=window)[:n], out[:n])
    pool.close()


@pytest.mark.parametrize("seed", range(10))
def test_prompt_batches(seed):
    rng = random.Random(100 + seed)
    new, before = _batch(rng)
    hq, hkv, d = rng.choice(HEADS)
    keys = None if rng.random() < 0.4 else [max(0, n + b - rng.choice([0, 0, 50])) for n, b in zip(new, before)]
    causal = rng.random() < 0.7
    run_prompt(seed, new, keys, hq, hkv, d, causal=causal, window=rng.choice([0, rng.randint(1, 300)]) if causal else 0)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_many_units_of_every_kind_many_times(kv):
    """More units of work than CTAs take at once, some of one stream, some of both, some of the same rows in both:
    whatever their order in time, the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    new = [1, 40, 130, 2, 0, 70] * 40
    lens = [1 + n + (i * 37) % 300 for i, n in enumerate(new)]
    pool, tables = make_cache(gen, lens, 8, 64, kv)
    q = torch.randn(sum(new), 32, 64, generator=gen, device="cuda").to(torch.bfloat16)
    args = (q, tables, ints(lens), starts_of(new), 0.125, max(lens))
    out = pool.prefill(*args)
    check_prefill(pool, tables, q, out, new[:12], lens[:12], 0.125, 0, kv)
    for _ in range(20):
        assert torch.equal(pool.prefill(*args), out)
    assert pool.device_error() == 0
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("seed", range(4))
def test_short_calls_with_and_without_a_plan(kv, seed):
    """A bound on the lengths that is far above them makes a short call one with a plan."""
    rng = random.Random(seed + 50)
    new = [rng.choice([0, 1, 1, 2, 17, 40]) for _ in range(rng.randint(1, 12))]
    lens = [n + rng.choice([0, 5, 130, 600, 1400]) for n in new]
    hq, hkv, d = rng.choice([(8, 2, 128), (14, 2, 64), (4, 4, 64), (40, 1, 128)])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pool, tables = make_cache(gen, lens, hkv, d, kv)
    tables = torch.cat([tables, torch.full((len(new), 640), -1, dtype=torch.int32, device="cuda")], 1)
    q = (2 * torch.randn(max(1, sum(new)), hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
    for most in (max(lens), 10000):
        out = pool.prefill(q, tables, ints(lens), starts_of(new), d ** -0.5, most)
        assert pool.device_error() == 0
        check_prefill(pool, tables, q, out, new, lens, d ** -0.5, 0, (kv, seed, most))
        for _ in range(3):
            assert torch.equal(pool.prefill(q, tables, ints(lens), starts_of(new), d ** -0.5, most)[:sum(new)], out[:sum(new)])
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_one_long_context_among_thousands_of_units(kv):
    """A unit of work that is large beside a CTA's share, among more units than one pass of the plan takes."""
    gen = torch.Generator(device="cuda").manual_seed(10)
    new, lens = [1] * 400, [1 + (i * 29) % 60 for i in range(400)]
    new[217], lens[217] = 30, 20000
    pool, tables = make_cache(gen, lens, 8, 64, kv)
    q = torch.randn(sum(new), 16, 64, generator=gen, device="cuda").to(torch.bfloat16)
    out = pool.prefill(q, tables, ints(lens), starts_of(new), 0.125, 20000)
    assert pool.device_error() == 0
    check_prefill(pool, tables[210:225], q[210:254], out[210:254], new[210:225], lens[210:225], 0.125, 0, kv)
    check_prefill(pool, tables[:3], q[:3], out[:3], new[:3], lens[:3], 0.125, 0, kv)
    check_prefill(pool, tables[-3:], q[-3:], out[-3:], new[-3:], lens[-3:], 0.125, 0, kv)
    pool.close()


@pytest.mark.parametrize("seqs", [1024, 1025, 3000])
def test_more_sequences_than_the_plan_holds(seqs):
    gen = torch.Generator(device="cuda").manual_seed(11)
    new = [(i * 7) % 4 for i in range(seqs)]
    lens = [n + (i * 13) % 40 for i, n in enumerate(new)]
    pool, tables = make_cache(gen, lens, 1, 64, "bf16")
    q = torch.randn(sum(new), 4, 64, generator=gen, device="cuda").to(torch.bfloat16)
    out = pool.prefill(q, tables, ints(lens), starts_of(new), 0.125, 5 * 16)
    assert pool.device_error() == 0
    at = 0
    for b, n in enumerate(new):
        if b % 41 == 0 or b > seqs - 3:
            check_prefill(pool, tables[b:b + 1], q[at:at + n], out[at:at + n], [n], [lens[b]], 0.125, 0, b)
        at += n
    assert not out.isnan().any()
    pool.close()


def test_two_calls_at_once():
    """Two pools, two streams, two workspaces: calls that overlap on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    sides = []
    for kv, hkv, d in (("bf16", 4, 128), ("int8", 8, 64)):
        new, lens = [300, 1, 40], [900, 2000, 40]
        pool, tables = make_cache(gen, lens, hkv, d, kv)
        q = torch.randn(sum(new), 16, d, generator=gen, device="cuda").to(torch.bfloat16)
        args = (q, tables, ints(lens), starts_of(new), d ** -0.5, 2000)
        ws = torch.empty(pkv.prefill_workspace_bytes(pool, 3, 16, sum(new), 2000), dtype=torch.uint8, device="cuda")
        sides.append((pool, args, pool.prefill(*args), torch.empty_like(q), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for pool, args, _, out, ws, stream in sides:
            pool.prefill(*args, out=out, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for pool, _, expect, out, _, _ in sides:
        assert torch.equal(out, expect) and pool.device_error() == 0
        pool.close()
