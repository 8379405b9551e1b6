"""The schedule's scratch in the shared memory of the paged kernels, read from the
source: paged_range keeps a sum per warp and the two words of what it found, and
writes the table of sequences behind while the last of them may still be read."""
import os
import re

import pytest

from kv_cached_gqa_rope_gb300 import build
from test_launch_order_host import source

FILES = [f for f in sorted(os.listdir(build.CSRC)) if re.search(r"\bpaged_range<", source(f)) and f.endswith(".cu")]


def python(expr):
    """A constant expression of the sources, as Python's."""
    expr = re.sub(r"static_cast<int>", "", expr).replace("/", "//")
    while "?" in expr:  # (the innermost condition first)
        expr, n = re.subn(r"\(([^()?]+)\?([^():]+):([^():]+)\)", r"((\2) if (\1) else (\3))", expr)
        assert n, expr
    return expr


def constant(text, name, env):
    m = re.search(rf"constexpr int {name} = ([^;]+);", text)
    assert m, name
    return eval(python(m.group(1)), dict(env))


def test_the_users_are_found():
    assert {"paged_attention.cu", "paged_decode_e4m3.cu", "paged_mass.cu"} <= set(FILES)


@pytest.mark.parametrize("codes", [0, 1])
@pytest.mark.parametrize("file", FILES)
def test_scratch_has_its_room(file, codes):
    text = source(file)
    env = {"kE4M3": codes, "BM": 128}
    m = re.search(r"constexpr int paged_scratch_bytes\(int threads\) \{ return ([^;]+);", source("paged.cuh"))
    if m:
        env["paged_scratch_bytes"] = lambda threads: eval(python(m.group(1)), {"threads": threads})
    threads = constant(text, "THREADS", env)
    at = re.search(r"paged_range<THREADS>\([^;]*?C::(\w+_OFF)", text).group(1)
    # the constant that begins where the scratch ends
    after = re.search(rf"constexpr int \w+_OFF = {at} \+ ([^;]+);", text).group(1)
    room = eval(python(after), dict(env, THREADS=threads))
    assert room >= 4 * (threads // 32 + 2), f"{file}: {room} bytes for {threads // 32 + 2} ints"
