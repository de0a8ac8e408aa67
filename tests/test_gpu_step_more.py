"""The serving-step operators in calls that a program may make beside the ordinary ones: many steps in
place, memory of calls on another stream, outputs that cannot be."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("b,new,steps", [(40, 300, 12), (3, 1, 200), (1000, 7, 20)])
def test_many_steps_in_place(b, new, steps):
    """Lengths and the count of used blocks are replaced in place, by calls of one CTA and of several."""
    width = (new * steps + 31) // 16 + 1
    pool = pkv.PagedKVPool(b * width, 1, 64)
    free = torch.randperm(b * width, generator=torch.Generator().manual_seed(b)).to(torch.int32)
    tables = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    start = [(5 * i) % 17 for i in range(b)]  # lengths before the first step, 0 to 16 tokens: one block, if any
    used = 0
    host_tables = [[-1] * width for _ in range(b)]
    for i, t in enumerate(start):
        if t:
            host_tables[i][0] = int(free[used])
            used += 1
    tables.copy_(torch.tensor(host_tables, dtype=torch.int32))
    lens, count = _i32(start), _i32([used])
    got = []
    free_gpu = free.cuda()
    for _ in range(steps):
        out = pool.reserve_slots(tables, lens, torch.full((b,), new, dtype=torch.int32, device="cuda"), free_gpu,
                                 b * new, free_used=count, new_context_lens=lens, new_free_used=count)
        got.append((out[0], out[1]))
    free = free.tolist()
    host = list(start)
    for slots, pos in got:
        want_slots, want_pos = [], []
        for i in range(b):
            for t in range(host[i], host[i] + new):
                if t % 16 == 0:
                    host_tables[i][t // 16] = free[used]
                    used += 1
                want_slots.append(host_tables[i][t // 16] * 16 + t % 16)
                want_pos.append(t)
            host[i] += new
        assert slots.tolist() == want_slots and pos.tolist() == want_pos
    assert tables.tolist() == host_tables and lens.tolist() == host and count.item() == used
    assert pool.device_error() == 0
    pool.close()


def test_memory_made_for_a_call_on_another_stream():
    """Outputs that a call makes belong to its stream: what the current stream allocates and fills while
    the call still waits there does not touch them."""
    pool = pkv.PagedKVPool(64, 2, 128)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(200, 4, 128, device="cuda", generator=g).bfloat16()
    k, v = (torch.randn(200, 2, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    table = pkv.rope_table(512, 128)
    slots, pos = (torch.arange(200, dtype=torch.int32, device="cuda") for _ in range(2))
    ref = pool.norm_rope_and_cache(q, k, v, pos, slots, table)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = torch.full_like(q, 7.0)
    del junk  # its memory is the current stream's next block of this size
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    out = pool.norm_rope_and_cache(q, k, v, pos, slots, table, stream=side)
    tables, lens = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), _i32([0, 0])
    new, free = _i32([20, 30]), torch.arange(10, dtype=torch.int32, device="cuda")
    torch.cuda.current_stream().synchronize()
    res = pool.reserve_slots(tables, lens, new, free, 50, stream=side)
    made = pkv.rope_table(512, 128, stream=side)
    fill = [torch.full_like(q, -3.0), torch.full_like(table, -3.0)] + [torch.full((50,), 9, dtype=torch.int32, device="cuda")] * 6
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(made, table) and len(fill) == 8
    assert res[0].tolist() == list(range(20)) + list(range(32, 62))
    assert res[2].tolist() == [0, 20, 50] and res[3].tolist() == [20, 30] and res[4].tolist() == [4]
    assert pool.device_error() == 0
    pool.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["int8", "fp8"])
def test_codes_are_those_of_reshape_and_cache(kv, d):
    """Keys that are neither normalised nor rotated and values get the very codes and scales that
    reshape_and_cache writes: random rows, quotients on a tie of two codes and next to one, rows of
    tiny and of huge values, and rows with an infinity or a NaN."""
    g = torch.Generator().manual_seed(d)
    n, h = 4096, 2
    x = torch.randn(n, h, d, generator=g)
    x[512:1024] = (torch.randint(-254, 255, (512, h, d), generator=g) / 2.0).clamp(-127, 127)  # s = 1: halves are ties
    x[512:1024, :, 0] = 127.0
    x[1024:1536] = torch.randint(-448, 449, (512, h, d), generator=g).float()
    x[1024:1536, :, 0] = 448.0
    x[1536:2048] *= 2.0 ** torch.randint(-132, 120, (512, 1, 1), generator=g).float()
    x[2048:2560] = (x[2048:2560] * 8).round() / 8  # few different values: quotients fall together
    x = x.bfloat16()
    x[2560, 0, 3], x[2561, 1, 5], x[2562, 0, :2], x[2563] = float("inf"), float("nan"), float("-inf"), 0.0
    x = x.cuda()
    v = x.flip(0).contiguous()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    a, b = (pkv.PagedKVPool(n // 16, h, d, kv) for _ in range(2))
    a.reshape_and_cache(x, v, slots)
    b.norm_rope_and_cache(x, x, v, None, slots)
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
    for s, t in ((a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(s.view(torch.int32), t.view(torch.int32))
    for pool in (a, b):
        pool.close()


def test_queries_on_one_another_are_refused():
    pool = pkv.PagedKVPool(4, 2, 64)
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    k = torch.randn(3, 2, 64, device="cuda").bfloat16()
    slots = _i32([0, 1, 2])
    row = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PagedKVError):
        pool.norm_rope_and_cache(q, k, k, None, slots, out=row.expand(3, 4, 64))
    half = torch.zeros(2 * 4 * 64, dtype=torch.bfloat16, device="cuda").as_strided((3, 4, 64), (128, 64, 1))
    with pytest.raises(pkv.PagedKVError):
        pool.norm_rope_and_cache(q, k, k, None, slots, out=half)
    assert not row.any() and not half.any()
    # inputs may repeat: one token's queries for all, and one token by itself at any stride
    out = pool.norm_rope_and_cache(q[:1].expand(3, 4, 64), k, k, None, slots)
    assert torch.equal(out, q[:1].expand(3, 4, 64))
    assert torch.equal(pool.norm_rope_and_cache(q[:1], k[:1], k[:1], None, slots[:1], out=row), q[:1])
    assert pool.device_error() == 0
    pool.close()
