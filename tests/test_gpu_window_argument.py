"""Windows and lengths beyond 32 bits: no window is cut down to its low bits."""

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import build
from prompt_reference import ints, starts_of
from test_gpu_prompt import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70])
def test_a_window_of_any_size(window):
    gen = torch.Generator(device="cuda").manual_seed(1)
    new, lens = [3, 40], [100, 40]
    pool, tables = make_cache(gen, lens, 2, 64, "bf16")
    q = torch.randn(sum(new), 4, 64, generator=gen, device="cuda").to(torch.bfloat16)
    args = (tables, ints(lens), starts_of(new), 0.125, 100)
    assert torch.equal(pool.prefill(q, *args, window=window), pool.prefill(q, *args))
    k = torch.randn(sum(new), 2, 64, generator=gen, device="cuda").to(torch.bfloat16)
    assert torch.equal(pool.prompt_attention(q, k, k, starts_of(new), 0.125, window=window),
                       pool.prompt_attention(q, k, k, starts_of(new), 0.125))
    one = (q[:2].contiguous(), tables, ints(lens), 0.125, 100)
    assert torch.equal(pool.decode(*one, window=window), pool.decode(*one))
    pool.close()


@pytest.mark.parametrize("window", [-1, -2 ** 31, -2 ** 32 + 5, -2 ** 70])
def test_negative_windows_are_refused(window):
    gen = torch.Generator(device="cuda").manual_seed(2)
    pool, tables = make_cache(gen, [100, 40], 2, 64, "bf16")
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PagedKVError):
        pool.prefill(q, tables, ints([100, 40]), starts_of([3, 2]), 0.125, 100, window=window)
    with pytest.raises(pkv.PagedKVError):
        pool.prompt_attention(q, q[:, :2], q[:, 2:], starts_of([3, 2]), 0.125, window=window)
    with pytest.raises(pkv.PagedKVError):
        pool.decode(q[:2].contiguous(), tables, ints([100, 40]), 0.125, 100, window=window)
    pool.close()


@pytest.mark.parametrize("most", [2 ** 31 + 64, 2 ** 32 + 96, -2 ** 32 + 96])
def test_lengths_beyond_32_bits_are_refused(most):
    """Their low bits would be lengths that the tables hold."""
    pool = pkv.PagedKVPool(8, 2, 64, "bf16", fill=0)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    tables = ints([[0, 1, 2, 3, 4, 5, 6]])
    before = pkv.launch_count()
    with pytest.raises(pkv.PagedKVError):
        pkv.prefill_workspace_bytes(pool, 1, 4, 5, most)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PagedKVError):
        pool.prefill(q, tables, ints([96]), ints([0, 5]), 0.125, most, workspace=ws)
    assert pkv.launch_count() == before
    pool.close()
