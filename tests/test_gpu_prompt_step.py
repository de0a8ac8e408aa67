"""The prompt operators as a step uses them, all on the GPU: slots reserved from the lengths, queries and keys
normalised, rotated and cached, attention of chunks and single tokens over the cache in a captured step; the first
chunk's attention straight from the projection; the cache read back in front of new keys."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import attend, cached, check, ints, starts_of
from test_gpu_prompt import check_prefill, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_chunked_prompts_and_decodes_in_one_graph(kv):
    hq, hkv, d, seqs, most = 8, 2, 128, 4, 96
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool = pkv.PagedKVPool(200, hkv, d, kv, fill=0)
    table = pkv.rope_table(2048, d)
    qw, kw = ((1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    tables = torch.full((seqs, 64), -1, **i32)
    lens, new = torch.zeros(seqs, **i32), torch.zeros(seqs, **i32)
    free, used = torch.randperm(200, generator=gen, device="cuda").to(torch.int32), torch.zeros(1, **i32)
    slots, pos, qs = torch.empty(most, **i32), torch.empty(most, **i32), torch.empty(seqs + 1, **i32)
    qkv = torch.empty(most, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    q, out = (torch.empty(most, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(pkv.prefill_workspace_bytes(pool, seqs, hq, most, 1024), dtype=torch.uint8, device="cuda")

    def step():
        pool.reserve_slots(tables, lens, new, free, most, free_used=used, slot_mapping=slots, positions=pos, query_starts=qs,
                           new_context_lens=lens, new_free_used=used)
        pool.norm_rope_and_cache(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, slots, table, qw, kw, out=q)
        pool.prefill(q, tables, lens, qs, d ** -0.5, 1024, out=out, workspace=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    total = [0] * seqs
    for counts in ([50, 0, 0, 0], [46, 20, 1, 0], [1, 1, 1, 70], [1, 60, 1, 1], [0, 0, 0, 0], [1, 1, 1, 1], [30, 30, 30, 6]):
        new.copy_(ints(counts))
        qkv.normal_(generator=gen)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert pool.device_error() == 0
        total = [a + b for a, b in zip(total, counts)]
        assert lens.tolist() == total and qs.tolist() == starts_of(counts).tolist()
        check_prefill(pool, tables, q, out, counts, total, d ** -0.5, 0, (kv, counts))
        assert (out[sum(counts):] == 7.0).all()
        if all(c == 1 for c in counts):  # the decode sees the same
            other = pool.decode(q[:seqs].contiguous(), tables, lens, d ** -0.5, 1024)
            assert ((other.double() - out[:seqs].double()).abs() <= 2.0 ** -5 * (1 + out[:seqs].double().abs())).all()
    pool.close()


def test_first_chunk_from_the_projection_equals_the_cache():
    """A bf16 pool holds what was written: the packed call and the call over the cache see the same values."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = [33, 200, 1, 128]
    hq, hkv, d = 16, 4, 64
    x = torch.randn(sum(new), hq + 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    pool, tables = make_cache(gen, new, hkv, d, "bf16")
    slots = torch.cat([tables[b, torch.arange(n, device="cuda") // 16] * 16 + torch.arange(n, device="cuda", dtype=torch.int32) % 16
                       for b, n in enumerate(new)]).to(torch.int32)
    pool.reshape_and_cache(k.contiguous(), v.contiguous(), slots)
    a = pool.prompt_attention(q, k, v, starts_of(new), 0.125)
    b = pool.prefill(q, tables, ints(new), starts_of(new), 0.125, max(new))
    assert torch.equal(a, b)
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_cache_read_back_in_front_of_new_keys(kv):
    """gather_cache's rows with the new tokens' behind them, attended to by prompt_attention."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    before, new = [100, 0, 333], [20, 40, 1]
    hq, hkv, d = 8, 2, 128
    pool, tables = make_cache(gen, before, hkv, d, kv)
    total = [a + b for a, b in zip(before, new)]
    n, m = sum(new), sum(total)
    x = torch.randn(n, hq + 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
    keys, values = (torch.empty(m, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = row = 0
    for b, (t, c) in enumerate(zip(before, new)):  # each sequence's cached rows go where its keys start
        pool.gather_cache(tables[b:b + 1], ints([at, at + t]), m, k=keys, v=values)
        keys[at + t:at + t + c] = x[row:row + c, hq:hq + hkv]
        values[at + t:at + t + c] = x[row:row + c, hq + hkv:]
        at, row = at + t + c, row + c
    out = pool.prompt_attention(x[:, :hq], keys, values, starts_of(new), d ** -0.5, key_starts=starts_of(total))
    assert pool.device_error() == 0
    row = 0
    for b, (t, c) in enumerate(zip(before, new)):
        k, v, _ = cached(pool, tables[b], t)
        k, v = (y.to(torch.bfloat16).double() for y in (k, v))  # as gather_cache rounds them
        k = torch.cat([k, x[row:row + c, hq:hq + hkv].double()])
        v = torch.cat([v, x[row:row + c, hq + hkv:].double()])
        check(out[row:row + c], *attend(x[row:row + c, :hq].double(), k, v, d ** -0.5), t + c, (kv, b))
        row += c
    pool.close()
