"""reserve_slots on the GPU against the block manager's append and a plain loop: tables, slots,
positions and lengths are whole numbers and have to be equal."""

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


def _plain(tables, lens, new, free, used, max_tokens):
    tables = [list(r) for r in tables]
    slots, pos, starts = [], [], [0]
    for b, (t, n) in enumerate(zip(lens, new)):
        for p in range(t, t + n):
            if p % 16 == 0:
                tables[b][p // 16] = free[used]
                used += 1
            slots.append(tables[b][p // 16] * 16 + p % 16)
            pos.append(p)
        starts.append(len(slots))
    pad = max_tokens - len(slots)
    return tables, slots + [-1] * pad, pos + [0] * pad, starts, [t + n for t, n in zip(lens, new)], used


def _case(lens, new, seed, spare=3, width=None, used=0):
    g = torch.Generator().manual_seed(seed)
    have = [(t + 15) // 16 for t in lens]
    need = [(t + n + 15) // 16 for t, n in zip(lens, new)]
    width = width or max(need + [1]) + 2
    total = sum(need) + spare + used
    ids = torch.randperm(total + 11, generator=g)[:total].tolist()
    tables, at = [], 0
    for h in have:
        tables.append(ids[at:at + h] + [-7] * (width - h))
        at += h
    return tables, ids[at:], total + 11


@pytest.mark.parametrize("lens,new,pad,used", [
    ([0], [1], 0, 0),
    ([15], [1], 0, 0),
    ([16], [1], 3, 2),
    ([0, 0, 0], [0, 0, 0], 5, 1),
    ([5, 0, 16, 31, 200], [0, 40, 16, 1, 0], 0, 0),
    ([100 * i % 777 for i in range(64)], [1] * 64, 0, 5),
    ([37 * i % 3000 for i in range(600)], [(i * 7) % 6 for i in range(600)], 100, 0),   # more than a CTA's threads
    ([0] * 5, [1, 4097, 16, 0, 33], 17, 0),
    ([3] * 33, [700] * 33, 0, 0),                                                       # several CTAs
    ([i % 40 for i in range(5000)], [i % 3 for i in range(5000)], 9, 0),                # over 48 KB of shared memory
])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_a_plain_loop(lens, new, pad, used, in_place):
    tables, free, nb = _case(lens, new, seed=len(lens), used=used)
    max_tokens = sum(new) + pad
    expect = _plain(tables, lens, new, free, used, max_tokens)
    pool = pkv.PagedKVPool(nb, 1, 64, "bf16")
    tab, L, u = _i32(tables), _i32(lens), _i32([used])
    kw = dict(new_context_lens=L, new_free_used=u) if in_place else {}
    slots, pos, starts, after, now = pkv.reserve_slots(pool, tab, L, _i32(new), _i32(free), max_tokens, free_used=u, **kw)
    assert pool.device_error() == 0
    assert tab.tolist() == expect[0]
    assert slots.tolist() == expect[1] and pos.tolist() == expect[2] and starts.tolist() == expect[3]
    assert after.tolist() == expect[4] and now.tolist() == [expect[5]]
    if not in_place:
        assert L.tolist() == lens and u.tolist() == [used]
        again = pkv.reserve_slots(pool, tab, L, _i32(new), _i32(free), max_tokens, free_used=u)  # the same call once more
        assert again[0].tolist() == expect[1] and tab.tolist() == expect[0]
    pool.close()


@pytest.mark.parametrize("what", ["free", "table", "tokens", "negative length", "negative count", "used past the list",
                                  "negative used", "overflow"])
def test_all_or_nothing(what):
    lens, new = [5, 16, 40] + [0] * 20, [40, 3, 9] + [900] * 20
    tables, free, nb = _case(lens, new, seed=3, spare=0)
    max_tokens, used, expect = sum(new), 0, pkv.DEVERR_CAPACITY
    if what == "free":
        free = free[:-1]
    elif what == "table":
        tables = [r[:56] for r in tables]  # 900 tokens take 57 blocks
    elif what == "tokens":
        max_tokens -= 1
    elif what == "negative length":
        lens = [-1] + lens[1:]
        expect = pkv.DEVERR_CONTEXT_LEN
    elif what == "negative count":
        new = new[:-1] + [-4]
        expect = pkv.DEVERR_CONTEXT_LEN
    elif what == "used past the list":
        used = len(free) + 1
    elif what == "negative used":
        used = -1
    else:
        new = new[:3] + [2 ** 31 - 1] * 20
    pool = pkv.PagedKVPool(nb, 1, 64, "bf16")
    tab, L, u = _i32(tables), _i32(lens), _i32([used])
    slots, pos, starts, after, now = pkv.reserve_slots(pool, tab, L, _i32(new), _i32(free), max_tokens, free_used=u,
                                                       new_context_lens=L, new_free_used=u)
    assert pool.device_error() == expect
    assert tab.tolist() == tables and after.tolist() == lens and now.tolist() == [used]
    assert set(slots.tolist()) == {-1} and set(pos.tolist()) == {0} and set(starts.tolist()) == {0}
    # the pool serves the next call as if nothing had happened
    ok = pkv.reserve_slots(pool, _i32([[-1] * 4]), _i32([0]), _i32([33]), _i32([2, 0, 1]), 33)
    assert ok[0].tolist() == [2 * 16 + i for i in range(16)] + list(range(16)) + [16] and pool.device_error() == 0
    pool.close()


def test_block_ids_outside_the_pool():
    pool = pkv.PagedKVPool(4, 1, 64, "bf16")
    tab = _i32([[3, -1, -1], [9, -1, -1], [0, -1, -1]])  # the second one's partly filled block does not exist
    slots, *_ = pkv.reserve_slots(pool, tab, _i32([4, 4, 16]), _i32([2, 2, 2]), _i32([4]), 6)  # nor does the free one
    assert slots.tolist() == [3 * 16 + 4, 3 * 16 + 5, -1, -1, -1, -1]
    assert pool.device_error() == pkv.DEVERR_BLOCK_ID
    pool.close()


def test_same_slots_as_the_block_manager_over_many_steps():
    nb, n = 700, 12
    pool = pkv.PagedKVPool(nb, 2, 64, "bf16")
    bm = pkv.BlockManager(nb, max_seqs=n, max_blocks_per_seq=64)
    seqs = [bm.add_sequence() for _ in range(n)]
    free = bm.free_list(nb).cuda()
    tab = torch.full((n, 64), -1, dtype=torch.int32, device="cuda")
    L, u = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(8)
    for step in range(40):
        new = torch.randint(0, 90 if step % 10 == 0 else 3, (n,), generator=g).tolist()
        slots, pos, starts, _, _ = pkv.reserve_slots(pool, tab, L, _i32(new), free, max(1, sum(new)), free_used=u,
                                                     new_context_lens=L, new_free_used=u)
        expect, copies = bm.append(seqs, new)
        assert len(copies) == 0 and slots.tolist()[:sum(new)] == expect.tolist()
        table, lens = bm.tables(seqs)
        assert tab.tolist() == table.tolist() and L.tolist() == lens.tolist()
        assert u.item() == nb - bm.stats()[0]
    assert pool.device_error() == 0
    pool.close()


def test_empty_batch_and_refusals():
    pool = pkv.PagedKVPool(4, 1, 64, "bf16")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    slots, pos, starts, after, used = pkv.reserve_slots(pool, e.view(0, 4), e, e, e, 3)
    assert slots.tolist() == [-1] * 3 and starts.tolist() == [0] and used.tolist() == [0] and after.numel() == 0
    tab, one = _i32([[-1] * 4]), _i32([1])
    before = pkv.launch_count()
    for bad in (dict(num_new_tokens=_i32([1, 1])), dict(block_tables=_i32([[0], [0]])), dict(max_tokens=-1),
                dict(free_used=_i32([0, 0])), dict(query_starts=_i32([0])), dict(slot_mapping=_i32([0, 0])),
                dict(block_tables=tab.t()), dict(context_lens=one.cpu())):
        args = dict(block_tables=tab, context_lens=one, num_new_tokens=one, free_blocks=one, max_tokens=1) | bad
        with pytest.raises(ValueError):
            pkv.reserve_slots(pool, **args)
    with pytest.raises(pkv.PagedKVError):
        n = 16385
        z = torch.zeros(n, dtype=torch.int32, device="cuda")
        pkv.reserve_slots(pool, z.view(n, 1), z, z, one, 1)
    with pytest.raises(pkv.PagedKVError):
        pkv.reserve_slots(pool, torch.empty(1, 0, dtype=torch.int32, device="cuda"), one, one, one, 1)
    assert pkv.launch_count() == before
    pool.close()
