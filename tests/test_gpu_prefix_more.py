"""shared_prefix_decode where it could go wrong beside its arithmetic: repeated calls, many pieces of
work, pools past 32-bit offsets, other streams, unusual scales.  The tolerance is that of
test_gpu_prefix."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("kv,d,hq,hkv,groups", [
    ("bf16", 128, 32, 32, [(128 * (1 + i % 7) + 16 * i, [1 + j for j in range(1 + i % 6)]) for i in range(16)]),
    ("bf16", 128, 32, 4, [(1024, [9] * 40), (272, [3] * 17), (2000, [1] * 5)]),      # both ways of sharing tiles out
    ("int8", 128, 32, 4, [(1024, [9] * 40), (272, [3] * 17), (2000, [1] * 5)]),
    ("fp8", 64, 16, 16, [(16 * (1 + 5 * i), [2, 3, 4]) for i in range(50)]),         # more than 32 groups
    ("bf16", 64, 32, 2, [(640, [1 + i % 9 for i in range(60)])] + [(48, [5, 6])] * 40),
])
def test_many_calls_give_the_same_bits(kv, d, hq, hkv, groups):
    """Pieces of work begin and end at other moments in every call; nothing may depend on that."""
    x = Batch(groups, hq, hkv, d, kv, seed=2)
    ws = torch.full((pkv.shared_prefix_workspace_bytes(x.pool, x.b, hq, len(groups), x.max_prefix, x.max_own),), 255,
                    dtype=torch.uint8, device="cuda")
    ref = x.run(workspace=ws).clone()
    x.check(ref, seqs=range(0, x.b, max(1, x.b // 24)))
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        out = x.run(workspace=ws)
        bad += (out != ref).sum()
    assert bad.item() == 0 and x.pool.device_error() == 0
    x.pool.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_pool_past_32_bit_offsets(kv):
    """K and V of more than 2^31 values each, blocks from all over them."""
    x = Batch([(1040, [40, 3, 60]), (160, [100])], 8, 1, 128, kv, seed=7, spare=1_150_000)
    assert x.pool.k_cache.numel() > 2 ** 31 and int(x.tables[x.tables < x.pool.num_blocks].max()) * 16 * 128 > 2 ** 31
    out = x.run()
    assert x.pool.device_error() == 0
    x.check(out)
    x.pool.close()


@pytest.mark.parametrize("kv,d,hq,k", [("bf16", 128, 1, 1), ("bf16", 128, 4, 1), ("bf16", 64, 7, 1), ("fp8", 64, 4, 4),
                                        ("int8", 128, 8, 2), ("bf16", 128, 16, 1), ("int8", 64, 2, 1)])
def test_many_partial_states_of_a_row(kv, d, hq, k):
    """One kv head and one long prefix, so that nearly every CTA leaves a state for each row; the groups
    behind it are empty.  The rows' states are joined by the items over the sequences' own tokens, and,
    where those are split, by the merge pass."""
    x = Batch([(20000 // 16 * 16, [40, 9, 300])] + [(0, [])] * 60 + [(16, [5])], hq, 1, d, kv, k=k, seed=13)
    for args in ({}, {"partition_blocks": 2}):
        launches = pkv.launch_count()
        out = x.run(**args)
        assert pkv.launch_count() - launches == (3 if args else 2)
        assert x.pool.device_error() == 0
        x.check(out)
    x.pool.close()


@pytest.mark.parametrize("scale", [0.0, -0.09, 0.5])
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_scales(kv, scale):
    """A negative scale turns the order of the logits round; with 0 all tokens weigh the same."""
    x = Batch([(400, [30, 7]), (144, [5])], 8, 2, 128, kv, seed=8)
    x.scale = scale
    out = x.run()
    assert x.pool.device_error() == 0
    x.check(out)
    x.pool.close()


def test_own_workspace_and_stream():
    x = Batch([(640, [30, 7, 90])], 16, 4, 128, "bf16", seed=9)
    ref = x.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = x.run()
    b = x.run(stream=side)
    side.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref) and x.pool.device_error() == 0
    x.pool.close()


def test_memory_made_for_a_call_on_another_stream():
    """The output and the workspace that a call makes belong to its stream: what the current stream
    allocates and fills while the call still waits there does not touch them."""
    x = Batch([(640, [30, 7, 90])], 16, 4, 128, "bf16", seed=9)
    ref = x.run()
    need = pkv.shared_prefix_workspace_bytes(x.pool, x.b, 16, 1, x.max_prefix, x.max_own)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    out = x.run(stream=side)
    fill = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert torch.equal(out, ref) and x.pool.device_error() == 0 and len(fill) == 4
    x.pool.close()


def test_two_pools_on_two_streams():
    """Calls on pools of their own may overlap."""
    xs = [Batch([(2048, [30 + i, 7, 90] * 4), (512, [3, 4])], 16, 4, 128, kv, seed=20 + i)
          for i, kv in enumerate(("bf16", "int8"))]
    refs = [x.run().clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, x in enumerate(xs):
            with torch.cuda.stream(streams[i]):
                outs[i].append(x.run())
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        assert all(torch.equal(o, refs[i]) for o in outs[i]) and x.pool.device_error() == 0
        x.pool.close()


def test_pool_over_the_callers_tensors():
    x = Batch([(320, [30, 7])], 8, 2, 128, "int8", seed=11)
    ref = x.run()
    other = pkv.PagedKVPool.from_tensors(x.pool.k_cache, x.pool.v_cache, x.pool.k_scale, x.pool.v_scale)
    assert (other.num_blocks, other.kv_heads, other.head_dim, other.dtype) == (x.pool.num_blocks, 2, 128, "int8")
    mine, x.pool = x.pool, other
    assert torch.equal(x.run(), ref)
    with pytest.raises(ValueError):
        pkv.PagedKVPool.from_tensors(other.k_cache, other.v_cache)
    with pytest.raises(ValueError):
        pkv.PagedKVPool.from_tensors(other.k_cache, other.v_cache[:1], other.k_scale, other.v_scale)
    with pytest.raises(TypeError):
        pkv.PagedKVPool.from_tensors(other.k_cache, other.v_cache.view(torch.uint8), other.k_scale, other.v_scale)
    with pytest.raises(pkv.PagedKVError):
        pkv.PagedKVPool.from_tensors(torch.zeros(2, 2, 16, 96, dtype=torch.bfloat16, device="cuda"),
                                     torch.zeros(2, 2, 16, 96, dtype=torch.bfloat16, device="cuda"))
    other.close()
    mine.close()
