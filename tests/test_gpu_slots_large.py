"""reserve_slots with sums past 32 bits: counts that each fit max_tokens and the table's width, and new
blocks that the free list has, but more new tokens than any slot mapping holds."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("counts", [
    [1 << 29] * 4,                      # one warp's sums meet at 2^30 and 2^30
    [1 << 29] * 2 + [0] * 30 + [1 << 29] * 2,   # two warps' sums do
    [1 << 29] * 8,                      # sums of two such
    [(1 << 29) - 1] * 3 + [7],          # 2^31 is not reached, the limit is
])
def test_token_sums_past_31_bits(counts):
    max_tokens, n = 1 << 29, len(counts)
    width = (max(counts) + 15) // 16
    pool = pkv.PagedKVPool(8, 1, 64, "bf16")
    i32 = dict(dtype=torch.int32, device="cuda")
    tables = torch.full((n, width), -9, **i32)
    lens, new, used = torch.zeros(n, **i32), torch.tensor(counts, **i32), torch.zeros(1, **i32)
    free = torch.arange(sum((c + 15) // 16 for c in counts), **i32)  # enough blocks, by number
    slots, pos, starts, after, now = pkv.reserve_slots(pool, tables, lens, new, free, max_tokens, free_used=used)
    assert pool.device_error() == pkv.DEVERR_CAPACITY
    assert after.tolist() == [0] * n and now.tolist() == [0] and starts.tolist() == [0] * (n + 1)
    assert int(slots.min()) == int(slots.max()) == -1 and int(pos.min()) == int(pos.max()) == 0
    assert int(tables.min()) == int(tables.max()) == -9
    pool.close()
