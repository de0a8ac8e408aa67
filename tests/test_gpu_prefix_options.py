"""pkv_shared_prefix_decode with every plan knob of its options, which apply to the pass over the sequences'
own tokens: kernel, schedule, ring shape and partition size, through the C ABI (the Python call offers the
partition size).  The tolerance is that of test_gpu_prefix; the CUDA-core kernel keeps its weights in
32 bits and stays within it."""

import ctypes

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import _lib, build
from test_gpu_prefix import GROUPS, Batch

pytestmark = pytest.mark.gpu

OK, INVALID_ARG, UNSUPPORTED = 0, 1, 2
CUDA_CORE, TENSOR_CORE = 1, 2
GRID, PERSISTENT = 1, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _call(x, **knobs):
    """(status, output) of one call; the status alone where the workspace size is refused."""
    lib = _lib.load()
    opt = _lib.DecodeOptions(num_queries=x.k, **knobs)
    n = ctypes.c_size_t()
    st = lib.pkv_shared_prefix_workspace_bytes(x.pool.handle, x.b, x.hq, x.lens.shape[0], x.max_prefix, x.max_own,
                                               ctypes.byref(opt), ctypes.byref(n))
    ws = torch.full((max(n.value, 16),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x.q, float("nan"))
    again = lib.pkv_shared_prefix_decode(
        x.pool.handle, x.q.data_ptr(), x.tables.data_ptr(), x.tables.shape[1], x.context.data_ptr(), x.b, x.hq,
        x.starts.data_ptr(), x.lens.data_ptr(), x.lens.shape[0], x.max_prefix, x.max_own, x.scale, out.data_ptr(),
        ws.data_ptr(), ws.numel(), ctypes.byref(opt), torch.cuda.current_stream().cuda_stream)
    assert again == st
    return st, out


def _shapes(kv, d):
    if kv == "bf16":
        return [(2, 1), (3, 1)] if d == 128 else [(3, 1), (2, 2)]
    return [(3, 1), (2, 1), (2, 2), (3, 2)] if d == 128 else [(2, 2), (3, 1)]


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("int8", 128), ("int8", 64), ("fp8", 128), ("fp8", 64)])
@pytest.mark.parametrize("name", ["mixed", "no own tokens", "many small groups", "no group"])
@pytest.mark.parametrize("hq,hkv,k", [(8, 2, 1), (6, 6, 1), (8, 2, 3), (20, 1, 1)])
def test_kernels_and_schedules(kv, d, name, hq, hkv, k):
    groups = [(p, [t + k - 1 for t in own]) for p, own in GROUPS[name]]
    x = Batch(groups, hq, hkv, d, kv, k, seed=hq + k)
    step = max(1, x.b // 8)
    for kernel in (CUDA_CORE, TENSOR_CORE):
        for schedule in (GRID, PERSISTENT):
            for partition in (0, 3):
                st, out = _call(x, kernel=kernel, schedule=schedule, partition_blocks=partition)
                assert st == OK and x.pool.device_error() == 0
                x.check(out, seqs=range(0, x.b, step))
    x.pool.close()


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("int8", 128), ("int8", 64), ("fp8", 128), ("fp8", 64)])
@pytest.mark.parametrize("hq,hkv,k", [(8, 2, 1), (32, 2, 1), (4, 2, 4)])
def test_ring_shapes(kv, d, hq, hkv, k):
    x = Batch([(400, [30 + k, k, 500]), (None, [k, 90])], hq, hkv, d, kv, k, seed=6)
    ran = 0
    for stages, bps in _shapes(kv, d):
        st, out = _call(x, kernel=TENSOR_CORE, stages=stages, blocks_per_stage=bps)
        assert st in (OK, UNSUPPORTED)  # not every shape holds 16 columns
        if st == OK:
            ran += 1
            assert x.pool.device_error() == 0
            x.check(out)
    assert ran >= (2 if hq * k // hkv <= 8 else 1)
    x.pool.close()


def test_refused_knobs():
    x = Batch([(160, [40, 1])], 8, 2, 128, "bf16", seed=4)
    before = pkv.launch_count()
    for bad, status in ((dict(kernel=3), INVALID_ARG), (dict(schedule=3), INVALID_ARG), (dict(window=64), UNSUPPORTED),
                        (dict(window=-1), INVALID_ARG), (dict(stages=7), UNSUPPORTED),
                        (dict(kernel=CUDA_CORE, stages=2), UNSUPPORTED)):
        assert _call(x, **bad)[0] == status, bad
    assert pkv.launch_count() == before
    x.pool.close()
