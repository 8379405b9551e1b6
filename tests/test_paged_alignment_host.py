"""Shared arrays that are read as 16-byte vectors say that they are aligned so:
nothing else promises it."""
import re

import pytest

from kv_cached_gqa_rope_gb300 import build
from test_launch_order_host import source


@pytest.mark.parametrize("file", build.SOURCES)
def test_shared_arrays_read_as_vectors_are_aligned(file):
    text = source(file)
    aligned = set(re.findall(r"struct\s+__align__\(16\)\s+(\w+)", text + source("rope_math.cuh")))
    for m in re.finditer(r"(?<!extern )__shared__\s+(__align__\(\d+\)\s+)?(\w+)\s+([^;]+);", text):
        align, kind, names = m.groups()
        if kind in aligned | {"float4", "uint4", "int4"} or (align and int(re.search(r"\d+", align).group()) >= 16):
            continue
        for name in re.findall(r"(\w+)\s*(?:\[[^\]]*\]\s*)+", names):
            assert not re.search(r"reinterpret_cast<(?:const )?(?:float4|uint4|int4)\*>\(\s*&?" + name + r"\b", text), \
                f"{file}: {name} is read 16 bytes at a time, its type promises less"
