"""Kernels' dynamic shared memory: units include several kernels' headers, and one name for arrays of different
alignment leaves it to the order of the headers which of them holds."""

import re
from pathlib import Path

CSRC = Path(__file__).resolve().parent.parent / "paged_kv_cache_264_gb300" / "csrc"


def test_a_name_has_one_alignment():
    found = {}
    for path in sorted(CSRC.iterdir()):
        if path.suffix in (".cu", ".cuh"):
            for align, name in re.findall(r"extern __shared__ (?:__align__\((\d+)\) )?[\w ]+? (\w+)\[\]", path.read_text()):
                found.setdefault(name, set()).add(align)
    assert found and all(len(a) == 1 for a in found.values()), found
