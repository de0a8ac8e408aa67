"""The host side of the serving-step operators, without a GPU: the block manager's free list
and prefix groups, the argument struct's layout, and refusals that touch no device."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import paged_kv_cache_264_gb300 as pkv
from paged_kv_cache_264_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_free_list_is_the_order_append_takes(lib):
    bm = pkv.BlockManager(40, max_seqs=4, max_blocks_per_seq=32)
    a, b = bm.add_sequence(), bm.add_sequence()
    bm.append([a, b], [70, 5])
    bm.truncate(a, 20)  # gives back three blocks, to be handed out next
    ids = bm.free_list(6)
    assert bm.free_list(6).tolist() == ids.tolist()  # nothing was taken
    slots, _ = bm.append([a, b], [44, 43])  # a: 20 -> 64 (2 blocks), b: 5 -> 48 (2 blocks)
    table, _ = bm.tables([a, b])
    assert table[0, 2:4].tolist() + table[1, 1:3].tolist() == ids[:4].tolist()
    assert bm.free_list(0).shape == (0,)
    with pytest.raises(pkv.PagedKVError):
        bm.free_list(bm.stats()[0] + 1)
    with pytest.raises(pkv.PagedKVError):
        bm.free_list(-1)


def test_prefix_groups(lib):
    bm = pkv.BlockManager(400, max_seqs=16, max_blocks_per_seq=40)
    p = bm.add_sequence()
    bm.append([p], [100])                       # 6 whole blocks and a partial one
    family = [p] + [bm.fork(p) for _ in range(3)]
    bm.append(family, [1] * 4)                  # the partial block is copied, the whole ones stay shared
    lone = bm.add_sequence()
    bm.append([lone], [33])
    q = bm.add_sequence()
    bm.append([q], [64])
    twin = bm.fork(q)
    starts, lens = bm.prefix_groups(family + [lone, q, twin])
    assert starts.tolist() == [0, 4, 5, 7]
    assert lens.tolist() == [96, 0, 64]         # whole blocks; a group of one shares nothing
    # every one of k queries has to see the whole prefix: 64 tokens, the first query sees 61
    assert bm.prefix_groups([q, twin], num_queries=4)[1].tolist() == [48]
    # joining must not lower what is saved: two sequences with 6 blocks in common, then one with 1
    r = bm.add_sequence()
    bm.append([r], [20])
    r1 = bm.fork(r)
    bm.append([r], [90])
    r2 = bm.fork(r)
    starts, lens = bm.prefix_groups([r, r2, r1])
    assert starts.tolist() == [0, 2, 3] and lens.tolist() == [96, 0]
    # released blocks are not shared
    bm.release_before(q, 32)
    assert bm.prefix_groups([q, twin])[1].tolist() == [0, 0]
    assert bm.prefix_groups([])[0].tolist() == [0]
    for bad in (0, 17):
        with pytest.raises(pkv.PagedKVError):
            bm.prefix_groups([q, twin], num_queries=bad)
    with pytest.raises(pkv.PagedKVError):
        bm.prefix_groups([15])


def test_norm_rope_struct_matches_the_header(tmp_path, lib):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f[0] for f in _lib.NormRope._fields_]
    consts = {"PKV_DEVERR_CAPACITY": pkv.DEVERR_CAPACITY, "PKV_DEVERR_POSITION": pkv.DEVERR_POSITION,
              "PKV_DEVERR_PREFIX": pkv.DEVERR_PREFIX}
    body = ['printf("size %zu\\n", sizeof(pkv_norm_rope));']
    body += [f'printf("{f} %zu\\n", offsetof(pkv_norm_rope, {f}));' for f in fields]
    body += [f'printf("{c} %lld\\n", (long long)({c}));' for c in consts]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"pagedkv.h\"\nint main(void) {\n"
                   + "\n".join(body) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                      check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(_lib.NormRope)
    for f in fields:
        assert int(got[f]) == getattr(_lib.NormRope, f).offset, f
    for c, v in consts.items():
        assert int(got[c]) == v


FAKE = ctypes.c_void_p(0x100000)  # aligned, never dereferenced


def test_null_pool_is_refused(lib):
    a = _lib.NormRope()
    n = ctypes.c_size_t()
    assert lib.pkv_norm_rope_and_cache(None, ctypes.byref(a), None) == _lib.PKV_ERR_INVALID_ARG
    assert lib.pkv_reserve_slots(None, FAKE, 4, FAKE, FAKE, 1, FAKE, 4, None, 1, FAKE, FAKE, FAKE, FAKE, FAKE,
                                 None) == _lib.PKV_ERR_INVALID_ARG
    assert lib.pkv_shared_prefix_decode(None, FAKE, FAKE, 4, FAKE, 1, 8, FAKE, FAKE, 1, 16, 16, 1.0, FAKE, FAKE,
                                        1 << 20, None, None) == _lib.PKV_ERR_INVALID_ARG
    assert lib.pkv_shared_prefix_workspace_bytes(None, 1, 8, 1, 16, 16, None, ctypes.byref(n)) == \
        _lib.PKV_ERR_INVALID_ARG


@pytest.mark.parametrize("args,expect", [
    ((None, 16, 64, 1e4), _lib.PKV_ERR_INVALID_ARG),
    ((FAKE, 0, 64, 1e4), _lib.PKV_ERR_INVALID_ARG),
    ((FAKE, 16, 0, 1e4), _lib.PKV_ERR_INVALID_ARG),
    ((FAKE, 16, 64, 0.0), _lib.PKV_ERR_INVALID_ARG),
    ((FAKE, 16, 64, float("nan")), _lib.PKV_ERR_INVALID_ARG),
    ((ctypes.c_void_p(0x100004), 16, 64, 1e4), _lib.PKV_ERR_INVALID_ARG),
    ((FAKE, 16, 24, 1e4), _lib.PKV_ERR_UNSUPPORTED),
])
def test_rope_table_refuses(lib, args, expect):
    assert lib.pkv_rope_table(*args, None) == expect


def test_python_refuses_before_the_library():
    """Wrong types and host tensors never reach the library (no GPU is needed to say so)."""
    class Pool:
        head_dim, kv_heads = 64, 2

    i32 = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.reserve_slots(Pool(), torch.zeros(2, 4, dtype=torch.int32), i32, i32, i32, 4)
    with pytest.raises(TypeError):
        pkv.reserve_slots(Pool(), torch.zeros(2, 4), i32, i32, i32, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.norm_rope_and_cache(Pool(), x, x, x, i32, i32)
    with pytest.raises(TypeError):
        pkv.norm_rope_and_cache(Pool(), x.float(), x, x, i32, i32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.shared_prefix_decode(Pool(), x, torch.zeros(2, 4, dtype=torch.int32), i32, i32, i32, 1.0, 16, 16)
    with pytest.raises(TypeError):
        pkv.PagedKVPool.from_tensors(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.PagedKVPool.from_tensors(*(torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16),) * 2)
