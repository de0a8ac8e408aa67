"""paged_attention_prefill over INT8 and FP8 pools of 2^31 rows of head_dim and more.  Their codes come by plain loads,
which have no limit there; a bf16 pool's tensor maps do."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import cached, ints, starts_of
from test_gpu_prompt import check_prefill

pytestmark = pytest.mark.gpu

HKV, D = 8, 64
BLOCKS = 2 ** 31 // (HKV * 16) + 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(scope="module")
def memory():
    """Codes and scales of such a pool; K and V share them, and only the blocks of the tables are ever touched."""
    torch.cuda.empty_cache()
    need = BLOCKS * HKV * 16 * (D + 4)
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip(f"{need >> 30} GiB of device memory")
    held = [torch.empty(BLOCKS, HKV, 16, D, dtype=torch.uint8, device="cuda"),
            torch.empty(BLOCKS, HKV, 16, dtype=torch.float32, device="cuda")]
    yield held
    held.clear()
    torch.cuda.empty_cache()  # other processes of the tests need it


@pytest.mark.parametrize("kv", ["int8", "fp8"])
def test_code_pools_of_two_to_the_31_rows(memory, kv):
    codes, scales = memory
    codes = codes.view(torch.int8) if kv == "int8" else codes
    pool = pkv.PagedKVPool.from_tensors(codes, codes, scales, scales)
    assert pool.num_blocks * HKV * 16 >= 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(len(kv))
    new, lens = [9, 70, 1], [200, 70, 2500]
    need = [(t + 15) // 16 for t in lens]
    # the first blocks and the last ones, in no order
    ids = torch.cat([torch.arange(sum(need) // 2, device="cuda"), BLOCKS - 1 - torch.arange(sum(need) - sum(need) // 2, device="cuda")])
    ids = ids[torch.randperm(len(ids), generator=gen, device="cuda")].to(torch.int32)
    tables = torch.full((3, 400), -1, dtype=torch.int32, device="cuda")
    for b, at in enumerate(starts_of(need)[:-1].tolist()):
        tables[b, :need[b]] = ids[at:at + need[b]]
    x = torch.randn(len(ids), HKV, 16, D, generator=gen, device="cuda")
    rows = (32 * x).round().clamp(-127, 127).to(torch.int8) if kv == "int8" else x.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[ids.long()] = rows
    scales[ids.long()] = torch.rand(len(ids), HKV, 16, generator=gen, device="cuda") / (32 if kv == "int8" else 1)
    q = torch.randn(sum(new), 16, D, generator=gen, device="cuda").to(torch.bfloat16)
    for most in (2500, 5000):
        out = pool.prefill(q, tables, ints(lens), starts_of(new), D ** -0.5, most)
        assert pool.device_error() == 0
        check_prefill(pool, tables, q, out, new, lens, D ** -0.5, 0, (kv, most))
    short = pool.prefill(q[:79], tables[:2], ints(lens[:2]), starts_of(new[:2]), D ** -0.5, 200)  # without a plan
    check_prefill(pool, tables, q[:79], short, new[:2], lens[:2], D ** -0.5, 0, (kv, "short"))
    k, v = pool.gather_cache(tables, starts_of(lens), sum(lens))
    at = 0
    for b, t in enumerate(lens):
        ref, _, _ = cached(pool, tables[b], t)
        assert ((k[at:at + t].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()
        at += t
    assert torch.equal(k, v) and pool.device_error() == 0
    pool.close()


def test_bf16_pools_of_two_to_the_31_rows_are_refused(memory):
    codes, _ = memory
    half = codes.view(torch.bfloat16)  # [BLOCKS, HKV, 16, D / 2]: as many values as BLOCKS / 2 blocks hold
    rows = half.view(-1)[:BLOCKS // 2 * HKV * 16 * D].view(BLOCKS // 2, HKV, 16, D)
    pool = pkv.PagedKVPool.from_tensors(rows, rows)
    q = torch.zeros(1, 16, D, dtype=torch.bfloat16, device="cuda")
    rows[0] = 0
    assert (pool.prefill(q, ints([[0]]), ints([1]), ints([0, 1]), 0.1, 16) == 0).all()  # half of the rows: taken
    # twice the blocks by the descriptor: refused before anything is read
    handle = pkv.pool_create(BLOCKS, HKV, D, "bf16", rows, rows)
    small, pool.handle = pool.handle, handle
    before = pkv.launch_count()
    with pytest.raises(pkv.PagedKVError):
        pool.prefill(q, ints([[0]]), ints([1]), ints([0, 1]), 0.1, 16)
    assert pkv.launch_count() == before
    pkv.pool_destroy(handle)
    pool.handle = small
    pool.close()
