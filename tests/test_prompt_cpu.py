"""The host side of prompt attention and cache read-back, without a GPU: the argument struct's layout
and refusals that touch no device."""

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


def test_prefill_struct_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f[0] for f in _lib.Prefill._fields_]
    body = ['printf("size %zu\\n", sizeof(pkv_prefill));']
    body += [f'printf("{f} %zu\\n", offsetof(pkv_prefill, {f}));' for f in fields]
    body += ['printf("deverr %u\\n", PKV_DEVERR_QUERY);']
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"pagedkv.h\"\nint main(void) {\n"
                   + "\n".join(body) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                      check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(_lib.Prefill)
    for f in fields:
        assert int(got[f]) == getattr(_lib.Prefill, f).offset, f
    assert int(got["deverr"]) == pkv.DEVERR_QUERY


def test_null_arguments_are_refused(lib):
    n = ctypes.c_size_t()
    a = _lib.Prefill()
    assert lib.pkv_prefill_workspace_bytes(None, 1, 4, 8, 16, ctypes.byref(n)) == _lib.PKV_ERR_INVALID_ARG
    assert lib.pkv_prefill_workspace_bytes(None, 1, 4, 8, 16, None) == _lib.PKV_ERR_INVALID_ARG
    assert lib.pkv_paged_attention_prefill(None, ctypes.byref(a), None) == _lib.PKV_ERR_INVALID_ARG
    assert lib.pkv_prompt_attention(None, None, None) == _lib.PKV_ERR_INVALID_ARG
    assert lib.pkv_gather_cache(None, None, 1, None, None, 1, 1, None, 64, None, 64, None) == _lib.PKV_ERR_INVALID_ARG


class _Pool:
    """What the argument checks look at, without a device."""

    kv_heads, head_dim, device_index, handle = 2, 64, 0, None

    class k_cache:
        device = torch.device("cuda", 0)


def test_tensors_on_the_host_are_refused():
    pool = _Pool()
    q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.prompt_attention(pool, q, k, k, i, 0.1)
    with pytest.raises(TypeError):
        pkv.prompt_attention(pool, q, k.float(), k, i, 0.1)
    with pytest.raises(ValueError):
        pkv.paged_attention_prefill(pool, q, i[None], i, i, 0.1, 16)
    with pytest.raises(TypeError):
        pkv.gather_cache(pool, k, i, 4)
    with pytest.raises(ValueError):
        pkv.gather_cache(pool, i[None], i, 4)
