"""A decode step as it is used, all of it on the GPU and captured once: slots reserved from the
lengths, queries and keys normalised, rotated and cached, attention over a shared prompt; several
replays in a row against 64-bit torch that keeps its own copy of every sequence."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _turn(x, w, table, pos):
    x = x.double()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    half = x.shape[-1] // 2
    c, s = table.double()[pos][:, None, :half], table.double()[pos][:, None, half:]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode_loop_in_one_graph(kv):
    hq, hkv, d, prompt, n, steps = 8, 2, 128, 150, 5, 20
    dev = torch.device("cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    pool = pkv.PagedKVPool(64, hkv, d, kv, fill=0)
    bm = pkv.BlockManager(64, max_seqs=8, max_blocks_per_seq=16)
    table = pkv.rope_table(512, d)
    qw, kw = ((1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))

    def projection(rows):
        return torch.randn(rows, hq + 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)

    def parts(x):
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    # the prompt, then forks; each gets its own copy of the partly filled block on its first token
    p = bm.add_sequence()
    slots, _ = bm.append([p], [prompt])
    x = projection(prompt)
    pos = torch.arange(prompt, dtype=torch.int32, device="cuda")
    pool.norm_rope_and_cache(*parts(x), pos, slots.cuda(), table, qw, kw)
    seqs = [p] + [bm.fork(p) for _ in range(n - 1)]
    first, copies = bm.append(seqs, [1] * n)
    pkv.copy_blocks(pool, copies.cuda())
    y = projection(n)
    pool.norm_rope_and_cache(*parts(y), torch.full((n,), prompt, dtype=torch.int32, device="cuda"), first.cuda(), table, qw, kw)
    history = [(torch.cat([x[:, hq:], y[i:i + 1, hq:]]), list(range(prompt + 1))) for i in range(n)]

    tables, lens = bm.tables(seqs)
    starts, prefix = bm.prefix_groups(seqs)
    assert starts.tolist() == [0, n] and prefix.tolist() == [prompt // 16 * 16]
    tables, lens, starts, prefix = (t.cuda() for t in (tables, lens, starts, prefix))
    free, used = bm.free_list(bm.stats()[0]).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    new = torch.ones(n, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device=dev)
    slots, pos, qs = torch.empty(n, **i32), torch.empty(n, **i32), torch.empty(n + 1, **i32)
    qkv = projection(n)
    q, out = torch.empty(n, hq, d, dtype=torch.bfloat16, device=dev), torch.empty(n, hq, d, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(pkv.shared_prefix_workspace_bytes(pool, n, hq, 1, 144, 64), dtype=torch.uint8, device=dev)

    def step():
        pool.reserve_slots(tables, lens, new, free, n, free_used=used, slot_mapping=slots, positions=pos, query_starts=qs,
                           new_context_lens=lens, new_free_used=used)
        pool.norm_rope_and_cache(*parts(qkv), pos, slots, table, qw, kw, out=q)
        pool.decode_shared_prefix(q, tables, lens, starts, prefix, d ** -0.5, 144, 64, out=out, workspace=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for i in range(steps):
        qkv.copy_(projection(n))
        graph.replay()
        torch.cuda.synchronize()
        assert pool.device_error() == 0
        expect, copied = bm.append(seqs, [1] * n)  # the host follows with the same counts
        assert len(copied) == 0 and slots.tolist() == expect.tolist()
        assert lens.tolist() == [prompt + 2 + i] * n and pos.tolist() == [prompt + 1 + i] * n
        for b in range(n):
            rows, at = history[b]
            history[b] = (torch.cat([rows, qkv[b:b + 1, hq:]]), at + [prompt + 1 + i])
            if i % 6 and i != steps - 1:
                continue
            rows, at = history[b]
            k = _turn(rows[:, :hkv], kw, table, torch.tensor(at, device=dev))
            v = rows[:, hkv:].double()
            qq = _turn(qkv[b:b + 1, :hq], qw, table, torch.tensor([prompt + 1 + i], device=dev))[0]
            s = torch.einsum("hgd,thd->hgt", qq.view(hkv, hq // hkv, d), k) * d ** -0.5
            w = torch.softmax(s, -1)
            ref = torch.einsum("hgt,thd->hgd", w, v).view(hq, d)
            wv = torch.einsum("hgt,thd->hgd", w, v.abs()).view(hq, d)
            # q and k are rounded (bf16: 2^-8 each; E4M3 keys: 2^-4), which moves a logit by at most
            # that share of sum |q k| * scale; the weights, the values' own rounding and the output follow
            kq = 2.0 ** -8 + (2.0 ** -8 if kv == "bf16" else 2.0 ** -4 + 2.0 ** -9)
            move = (torch.einsum("hgd,thd->hgt", qq.view(hkv, hq // hkv, d).abs(), k.abs()) * d ** -0.5 * kq).amax(-1)
            vq = 0.0 if kv == "bf16" else 2.0 ** -4 + 2.0 ** -9
            tol = (2 * torch.expm1(2 * move).clamp(max=4).reshape(hq, 1) + vq + 2.0 ** -7) * wv + 2.0 ** -7 * ref.abs()
            assert ((out[b].double() - ref).abs() <= tol).all()
            # and, tightly, against the pool's own contents
            dense = pool.decode(q[b:b + 1], tables[b:b + 1], lens[b:b + 1], d ** -0.5, int(lens[b]))
            assert ((dense[0].double() - out[b].double()).abs() <= 2 * (2.0 ** -8 * (2 * ref.abs() + wv) + 2.0 ** -10 * wv)
                    + 2.0 ** -7 * (dense[0].double() - ref).abs()).all()
    pool.close()
