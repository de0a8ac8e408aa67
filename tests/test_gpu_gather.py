"""gather_cache on the GPU.  A bf16 pool's values come back as they are; a quantised value is scale * code,
formed in fp32 (2^-24 of it) and rounded to bf16 (2^-8 of it)."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import cached, ints, starts_of
from test_gpu_prompt import make_cache

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
@pytest.mark.parametrize("hkv,d", [(1, 64), (2, 128), (8, 128), (5, 64)])
@pytest.mark.parametrize("lens,first", [([1], [0]), ([16, 17, 15], [0, 0, 0]), ([100, 0, 1, 300], [0, 40, 16, 33]),
                                        ([5] * 40, list(range(40))), ([2000], [77])])
def test_gather(lens, first, hkv, d, kv):
    gen = torch.Generator(device="cuda").manual_seed(len(lens) + d)
    pool, tables = make_cache(gen, [a + b for a, b in zip(lens, first)], hkv, d, kv)
    n = sum(lens)
    wide = torch.full((n + 4, hkv + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((n + 4, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k = wide[:, 1:]
    # a first row that is not 0: the rows before it are left too
    starts = starts_of(lens) + 2
    got = pool.gather_cache(tables, starts, n + 4, first_positions=ints(first), k=k, v=v)
    assert got[0] is k and got[1] is v
    at = 2
    for b, (t, f) in enumerate(zip(lens, first)):
        ref_k, ref_v, _ = cached(pool, tables[b], f + t)
        _check(k[at:at + t], ref_k[f:], kv, ("k", b))
        _check(v[at:at + t], ref_v[f:], kv, ("v", b))
        at += t
    for x in (k, v):
        assert (x[:2] == 7.0).all() and (x[at:] == 7.0).all()
    assert (wide[:, 0] == 7.0).all()
    if not any(first):
        k2, v2 = pool.gather_cache(tables, starts_of(lens), n)
        assert torch.equal(k2, k[2:at]) and torch.equal(v2, v[2:at])
    assert pool.device_error() == 0
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_gather_bad_blocks_and_positions(kv):
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool, tables = make_cache(gen, [100, 50], 2, 64, kv)
    good, _ = pool.gather_cache(tables, starts_of([100, 50]), 150)
    bad = tables.clone()
    bad[0, 1] = pool.num_blocks
    k, v = pool.gather_cache(bad, starts_of([100, 50]), 150)
    assert pool.device_error() == pkv.DEVERR_BLOCK_ID
    assert (k[16:32] == 0).all() and (v[16:32] == 0).all()
    assert torch.equal(k[:16], good[:16]) and torch.equal(k[32:], good[32:])
    # positions: past the table's row, and negative
    width = tables.shape[1] * 16
    k, _ = pool.gather_cache(tables, starts_of([3, 50]), 53, first_positions=ints([width - 1, 0]))
    assert pool.device_error() & pkv.DEVERR_CONTEXT_LEN
    assert (k[1:3] == 0).all() and torch.equal(k[3:], good[100:])
    k, _ = pool.gather_cache(tables, starts_of([3, 50]), 53, first_positions=ints([-2, 0]))
    assert pool.device_error() == pkv.DEVERR_CONTEXT_LEN
    assert (k[:3] == 0).all() and torch.equal(k[3:], good[100:])
    k, _ = pool.gather_cache(tables, starts_of([3, 50]), 53, first_positions=ints([2 ** 31 - 1, 0]))
    assert pool.device_error() == pkv.DEVERR_CONTEXT_LEN
    assert (k[:3] == 0).all()
    pool.close()


def test_gather_then_write_gives_the_cache_again():
    """Read back, written to other slots, read again: bf16 exactly; the codes of a quantised pool within a step."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    for kv in ("bf16", "int8", "fp8"):
        pool, tables = make_cache(gen, [333], 2, 128, kv)
        k, v = pool.gather_cache(tables, starts_of([333]), 333)
        other = pkv.PagedKVPool(30, 2, 128, kv, fill=0)
        pos = torch.arange(333, device="cuda", dtype=torch.int32)
        other.reshape_and_cache(k, v, pos)
        k2, v2 = other.gather_cache(torch.arange(21, device="cuda", dtype=torch.int32)[None], starts_of([333]), 333)
        if kv == "bf16":
            assert torch.equal(k, k2) and torch.equal(v, v2)
        else:
            # half a code's step of the row's largest value, and the roundings to bf16
            step = 1 / 254 if kv == "int8" else 2.0 ** -4
            for a, b in ((k, k2), (v, v2)):
                a, b = a.double(), b.double()
                assert ((a - b).abs() <= (step + 2.0 ** -8) * a.abs().amax(-1, keepdim=True) + 2.0 ** -8 * a.abs()).all()
        pool.close()
        other.close()


def test_gather_on_a_stream_and_in_a_graph():
    gen = torch.Generator(device="cuda").manual_seed(3)
    pool, tables = make_cache(gen, [64, 40], 2, 64, "fp8")
    starts = starts_of([64, 40])
    k, v = pool.gather_cache(tables, starts, 104)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k2, v2 = pool.gather_cache(tables, starts, 104, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    k3, v3 = torch.zeros_like(k), torch.zeros_like(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.gather_cache(tables, starts, 104, k=k3, v=v3)
    graph.replay()
    assert torch.equal(k, k3) and torch.equal(v, v3)
    pool.close()
