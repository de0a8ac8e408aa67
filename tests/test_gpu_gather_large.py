"""gather_cache where a CTA takes several tiles of 32 tokens, one after the other, and rows of tensors whose values lie
behind 2^31 elements.  A bf16 pool's values come back as they are; a quantised value is scale * code, formed in fp32
(2^-24 of it) and rounded to bf16 (2^-8 of it)."""

import random

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import cached, check, attend, ints, starts_of
from test_gpu_prompt import check_prefill, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _check(got, ref, kv, what):
    if kv == "bf16":
        assert torch.equal(got.double(), ref), what
    else:
        assert ((got.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all(), what


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128)])
def test_several_tiles_to_a_cta(hkv, d, kv):
    """At least three of them, the last not full, from a first row that is not 0; single tokens and empty sequences
    between long ones, each from a position of its own."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = random.Random(d)
    lens, room = [], 2 * 8 * sms * 32 + 1000
    while sum(lens) < room:
        lens.append(rng.choice([0, 1, 2, 31, 32, 33, rng.randint(3, 200), rng.randint(1000, 9000)]))
    lens[-1] += 32 - sum(lens) % 32 + 7  # 7 rows in the last tile
    first = [rng.choice([0, 0, 5, 16, rng.randint(1, 300)]) for _ in lens]
    gen = torch.Generator(device="cuda").manual_seed(hkv)
    pool, tables = make_cache(gen, [a + b for a, b in zip(lens, first)], hkv, d, kv)
    n, lead = sum(lens), 5
    k, v = (torch.full((n + lead + 4, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool.gather_cache(tables, starts_of(lens) + lead, n + lead + 4, first_positions=ints(first), k=k, v=v)
    assert pool.device_error() == 0
    at = lead
    for b, (t, f) in enumerate(zip(lens, first)):
        ref_k, ref_v, _ = cached(pool, tables[b], f + t)
        _check(k[at:at + t], ref_k[f:], kv, ("k", b))
        _check(v[at:at + t], ref_v[f:], kv, ("v", b))
        at += t
    for x in (k, v):
        assert (x[:lead] == 7.0).all() and (x[at:] == 7.0).all()
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_rows_behind_two_to_the_31_elements(kv):
    """Heads in the middle of wide rows: read back to there, and queries, keys, values and outputs that lie there."""
    hkv, d, width, t = 2, 64, 1024, 33000
    gen = torch.Generator(device="cuda").manual_seed(3)
    pool, tables = make_cache(gen, [t, 90], hkv, d, kv)
    wide = torch.zeros(t + 90, width, d, dtype=torch.bfloat16, device="cuda")
    assert wide[:t].numel() > 2 ** 31
    k, v = wide[:, 4:4 + hkv], wide[:, 10:10 + hkv]
    starts = starts_of([t, 90])
    pool.gather_cache(tables, starts, t + 90, k=k, v=v)
    for b, (lo, hi) in enumerate(((0, t), (t, t + 90))):
        for got, ref in zip((k, v), cached(pool, tables[b], hi - lo)):
            _check(got[lo:hi], ref, kv, b)
    assert (wide[:, :4] == 0).all() and (wide[:, 6:10] == 0).all()
    q, out = wide[:, 20:24], wide[:, 30:34]
    q.copy_(torch.randn(t + 90, 4, d, generator=gen, device="cuda"))
    # the last 90 rows as queries over keys in those rows, and over the cache
    mine = ints([t, t + 90])
    pool.prompt_attention(q, k, v, mine, 0.125, out=out)
    check(out[t:], *attend(q[t:].double(), k[t:].double(), v[t:].double(), 0.125), 90, "packed")
    assert (out[:t] == 0).all()
    out.zero_()
    pool.prefill(q, tables[1:], ints([90]), mine, 0.125, 90, out=out)
    check_prefill(pool, tables[1:], q[t:], out[t:], [90], [90], 0.125, 0, "cache")
    assert (out[:t] == 0).all() and pool.device_error() == 0
    pool.close()
