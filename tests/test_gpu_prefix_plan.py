"""How shared_prefix_decode plans the join of a row's states, seen by its launches: two where the items over
the sequences' own tokens join them, three with a merge pass; and the result of each plan, with the
tolerance of test_gpu_prefix."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _run(x, expect, step=1, **bounds):
    launches = pkv.launch_count()
    out = x.run(**bounds)
    assert pkv.launch_count() - launches == expect
    assert x.pool.device_error() == 0
    x.check(out, seqs=range(0, x.b, step))
    return out


def _padded(n, prefix=8192):
    """One long prefix of four sequences beside many groups of one block: each of its rows has a state from
    nearly every CTA, however many groups there are."""
    return [(prefix, [40, 9, 30, 17])] + [(16, [5 + i % 40 for i in range(8)])] * ((n - 4) // 8)


def test_long_prefix_beside_many_tiny_groups():
    """16 columns to an item, and more items than two an SM: up to 65 states of a row go to a merge pass, up
    to 13 do not."""
    for prefix, expect in ((8192, 3), (1536, 2)):
        x = Batch(_padded(300, prefix), 16, 1, 128, "bf16", seed=3)
        _run(x, expect, step=7)
        x.pool.close()


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("int8", 128), ("fp8", 128), ("bf16", 64), ("fp8", 64)])
@pytest.mark.parametrize("hq,hkv,k,n", [(16, 1, 1, 4), (16, 1, 1, 36), (12, 1, 1, 12), (32, 2, 1, 20), (7, 1, 3, 20), (40, 1, 1, 4),
                                        (24, 2, 4, 12)])
def test_items_of_fewer_columns(kv, d, hq, hkv, k, n):
    """Few items: their columns are shared out to more, the last one's part of them unused."""
    x = Batch(_padded(n, 2048), hq, hkv, d, kv, k, seed=n)
    out = _run(x, 2, step=3)
    assert torch.equal(x.run(), out)
    _run(x, 3, step=3, partition_blocks=1)
    x.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "int8", "fp8"])
def test_own_parts_around_one_items_length(kv):
    for own, expect in ((512, 2), (513, 2), (768, 2), (769, 3)):
        x = Batch([(1024, [own, 3, own - 5, 1])], 32, 8, 128, kv, seed=own)
        _run(x, expect)
        x.pool.close()


def test_bounds_given_as_capacities():
    """A captured step passes what its buffers hold, not what a batch needs."""
    x = Batch([(1024, [40, 9, 300]), (48, [7])], 32, 8, 128, "bf16", seed=1)
    _run(x, 2)
    width = (x.tables.shape[1] + 200) // 4 * 4
    tables = torch.full((x.b, width), -1, dtype=torch.int32, device="cuda")
    tables[:, :x.tables.shape[1]] = x.tables
    for mp, mo in ((width * 16, 300), (1024, width * 16), (width * 16, width * 16)):
        x.check(x.run(block_tables=tables, max_prefix_len=mp, max_suffix_len=mo))
    assert x.pool.device_error() == 0
    x.pool.close()
