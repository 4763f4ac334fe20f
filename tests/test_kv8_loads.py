"""Which loads the 8-bit attention may take through the read-only path.

That path (ld.global.nc) is for data that nobody writes while the kernel runs.  In a step the
attention kernel is resident while the append still writes the cache (it waits for it),
so what the append writes -- keys, values, scales, the rotated queries -- comes by
ordinary or L2 loads behind the wait; the page table, which no kernel of a step
writes, need not."""
import pathlib
import re

import pytest

SRC = pathlib.Path(__file__).resolve().parent.parent / "paged_kv_decode_16_gb300" / "csrc"


@pytest.mark.parametrize("name", ["kv8_decode.cuh", "kv8_umma.cu", "kv8_combine.cu",
                                  "kv8_plan.cuh"])
def test_no_read_only_loads_of_the_cache(name):
    text = re.sub(r"//[^\n]*", "", (SRC / name).read_text())
    for arg in re.findall(r"__ldg\(([^;]*)\)", text):
        assert "p.table" in arg, arg
    assert not re.search(r"ld\.global\.nc|__restrict__", text)
