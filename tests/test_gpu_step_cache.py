"""A captured decode step (slots reserved, queries and keys normalised, rotated and cached, attention over a
shared prompt) checked link by link against 64 bits on the CPU: the queries, what the pool holds at every
sequence's slots, and the attention over exactly what it holds.  So each tolerance is that of one link:
queries and cached rows those of test_gpu_rope (half a step of the type they are rounded to, and 2^-18 of
the pair's size for the 32-bit arithmetic), attention that of test_gpu_prefix."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build

pytestmark = pytest.mark.gpu

HQ, HKV, D, PROMPT, N, STEPS = 8, 2, 128, 150, 5, 14


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _turned(x, w, table, pos):
    """(norm and rotation of rows [t, h, D] at positions pos, size of each value's pair) in 64 bits."""
    x = x.double()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    c, s = (t[pos][:, None] for t in table.double().split(D // 2, 1))
    a, b = x.split(D // 2, 2)
    size = a.abs() + b.abs()
    return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([size, size], -1)


def _bf16_ok(got, ref, size):
    return bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size).all())


def _rows_ok(kv, codes, scale, ref, size):
    """Whether cached rows [t, h, D] stand for ref."""
    if kv == "bf16":
        return _bf16_ok(codes, ref, size)
    top = 127.0 if kv == "int8" else 448.0
    amax, s = ref.abs().amax(-1), scale.double()
    if not ((s - amax / top).abs() <= (2.0 ** -18 * size.amax(-1) + 2.0 ** -24 * amax) / top).all():
        return False
    half = 0.5 * s[..., None].expand_as(ref) if kv == "int8" else torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * s[..., None])
    tol = half * (1 + 2.0 ** -16) + 2.0 ** -17 * (size + amax[..., None])
    return bool(((codes.double() * s[..., None] - ref).abs() <= tol).all())


def _attention_ok(got, q, k, v):
    """Whether got [HQ, D] is the attention of q over k and v [t, HKV, D]."""
    x = torch.einsum("hgd,thd->hgt", q.view(HKV, HQ // HKV, D), k) * D ** -0.5
    w = torch.softmax(x, -1)
    ref = torch.einsum("hgt,thd->hgd", w, v).reshape(HQ, D)
    wv = torch.einsum("hgt,thd->hgd", w, v.abs()).reshape(HQ, D)
    return bool(((got.double() - ref).abs() <= 2.0 ** -8 * (2 * ref.abs() + wv) + 2.0 ** -11 * wv).all())


def _pool_rows(pool, name, slots):
    """(codes as numbers, scales or None) of the pool's rows at slots."""
    cache, scale = (pool.k_cache, pool.k_scale) if name == "k" else (pool.v_cache, pool.v_scale)
    blk, at = slots // 16, slots % 16
    rows = cache.cpu()[blk, :, at]
    rows = rows.view(torch.float8_e4m3fn).float() if pool.dtype == "fp8" else rows
    return rows, None if scale is None else scale.cpu()[blk, :, at]


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_every_link_of_a_captured_step(kv):
    gen = torch.Generator(device="cuda").manual_seed(17)
    pool = pkv.PagedKVPool(64, HKV, D, kv, fill=0)
    bm = pkv.BlockManager(64, max_seqs=8, max_blocks_per_seq=16)
    table = pkv.rope_table(512, D)
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))

    def projection(rows):
        return torch.randn(rows, HQ + 2 * HKV, D, generator=gen, device="cuda").to(torch.bfloat16)

    def parts(x):
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    p = bm.add_sequence()
    slots, _ = bm.append([p], [PROMPT])
    x = projection(PROMPT)
    pool.norm_rope_and_cache(*parts(x), torch.arange(PROMPT, dtype=torch.int32, device="cuda"), slots.cuda(), table, qw, kw)
    seqs = [p] + [bm.fork(p) for _ in range(N - 1)]
    first, copies = bm.append(seqs, [1] * N)
    pkv.copy_blocks(pool, copies.cuda())
    y = projection(N)
    pool.norm_rope_and_cache(*parts(y), torch.full((N,), PROMPT, dtype=torch.int32, device="cuda"), first.cuda(), table, qw, kw)
    history = [torch.cat([x[:, HQ:], y[i:i + 1, HQ:]]).cpu() for i in range(N)]

    tables, lens = (t.cuda() for t in bm.tables(seqs))
    starts, prefix = (t.cuda() for t in bm.prefix_groups(seqs))
    free, used = bm.free_list(bm.stats()[0]).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    new = torch.ones(N, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    slots, pos, qs = torch.empty(N, **i32), torch.empty(N, **i32), torch.empty(N + 1, **i32)
    qkv = projection(N)
    q, out = (torch.empty(N, HQ, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(pkv.shared_prefix_workspace_bytes(pool, N, HQ, 1, 144, 64), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pool.reserve_slots(tables, lens, new, free, N, free_used=used, slot_mapping=slots, positions=pos, query_starts=qs,
                           new_context_lens=lens, new_free_used=used)
        pool.norm_rope_and_cache(*parts(qkv), pos, slots, table, qw, kw, out=q)
        pool.decode_shared_prefix(q, tables, lens, starts, prefix, D ** -0.5, 144, 64, out=out, workspace=ws)

    table, qw, kw = table.cpu(), qw.cpu(), kw.cpu()
    for step in range(STEPS):
        qkv.copy_(projection(N))
        graph.replay()
        torch.cuda.synchronize()
        assert pool.device_error() == 0
        bm.append(seqs, [1] * N)  # the host follows with the same counts
        rows = bm.tables(seqs)[0]
        now = qkv.cpu()
        total = PROMPT + 2 + step
        for b in range(N):
            history[b] = torch.cat([history[b], now[b:b + 1, HQ:]])
            if step % 5 and step != STEPS - 1:
                continue
            at = torch.arange(total)
            where = rows[b, at // 16].long() * 16 + at % 16
            (kc, ks), (vc, vs) = (_pool_rows(pool, name, where) for name in "kv")
            k, ksize = _turned(history[b][:, :HKV], kw, table, at)
            v = history[b][:, HKV:].double()
            assert _rows_ok(kv, kc, ks, k, ksize) and _rows_ok(kv, vc, vs, v, v.abs())
            ref, size = _turned(now[b:b + 1, :HQ], qw, table, torch.tensor([total - 1]))
            got_q = q[b].cpu()
            assert _bf16_ok(got_q, ref[0], size[0])
            held_k = kc.double() * (1.0 if ks is None else ks.double()[..., None])
            held_v = vc.double() * (1.0 if vs is None else vs.double()[..., None])
            got = out[b].cpu()
            assert _attention_ok(got, got_q.double(), held_k, held_v)
            # these comparisons see mistakes: a position one off, two tokens' keys changed over, one value row lost
            wrong, wsize = _turned(history[b][:, :HKV], kw, table, at + 1)
            assert not _rows_ok(kv, kc, ks, wrong, wsize)
            assert not _bf16_ok(got_q, _turned(now[b:b + 1, :HQ], qw, table, torch.tensor([total]))[0][0], size[0])
            w = torch.softmax(torch.einsum("hgd,thd->hgt", got_q.double().view(HKV, HQ // HKV, D), held_k) * D ** -0.5, -1)
            top = int(w.sum((0, 1)).argmax())
            other = (top + 7) % total
            swapped = held_k.clone()
            swapped[[top, other]] = held_k[[other, top]]
            assert not _attention_ok(got, got_q.double(), swapped, held_v)
            lost = held_v.clone()
            lost[top] = 0
            assert not _attention_ok(got, got_q.double(), held_k, lost)
    pool.close()
