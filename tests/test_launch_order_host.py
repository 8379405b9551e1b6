"""Kernels launched with programmatic stream serialization wait for their
predecessor on every path.

Such a kernel may start while its predecessor still runs, and the wait of the
kernel behind it covers only its own direct predecessor.  A grid that ends
without having waited therefore lets its successor pass the grid before it.
Read from the source: the order of two grids that do not wait cannot be forced
in a run."""
import os
import re

import pytest

from kv_cached_gqa_rope_gb300 import build

KERNEL = re.compile(r"__global__ void\s+(?:__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(")


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


def kernels(text):
    """(name, body) of every kernel."""
    for m in KERNEL.finditer(text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield m.group(1), text[at:end]


def unwaited_returns(body):
    """The returns of a kernel that no wait precedes: neither one directly in
    front, nor one that the kernel's outermost block passes unconditionally."""
    depth, waited, bad = 0, False, []
    for m in re.finditer(r"[{}]|\breturn;|\bpdl_wait\(\);", body):
        t = m.group()
        before = body[:m.start()].rstrip()
        if t == "{":
            depth += 1
        elif t == "}":
            depth -= 1
        elif t == "pdl_wait();":
            waited = waited or (depth == 1 and before[-1] in ";{}")
        elif not waited and not before.endswith("pdl_wait();"):
            bad.append(" ".join(body[max(0, m.start() - 60):m.end()].split()))
    return bad, waited


FILES = [f for f in build.SOURCES if "programmaticStreamSerializationAllowed" in source(f)]
KERNELS = [(f, n) for f in FILES for n, _ in kernels(source(f))]


def test_the_kernels_are_found():
    names = {n for _, n in KERNELS}
    assert {"paged_rope_kv_store_kernel", "paged_attention_kernel", "paged_merge_kernel", "paged_mass_kernel",
            "paged_evict_select_kernel", "paged_evict_move_kernel", "prefill_attention_kernel",
            "rope_kv_store_kernel"} <= names


@pytest.mark.parametrize("file,name", [x for x in KERNELS if x[1] != "flash_decode_splitk_kernel"])
def test_every_path_waits(file, name):
    bad, waited = unwaited_returns(dict(kernels(source(file)))[name])
    assert not bad, f"{name} returns without waiting for the kernel before it: {bad}"
    assert waited, f"{name} does not wait for the kernel before it on every path"


@pytest.mark.parametrize("file,name", [x for x in KERNELS if "tmem_alloc(" in dict(kernels(source(x[0])))[x[1]]])
def test_no_grid_holds_tensor_memory_while_it_waits(file, name):
    """It could be what the CTAs it waits for still ask for.  (The decode step's
    early start does: the kernel it waits for is its own store, which has none.)"""
    body = dict(kernels(source(file)))[name]
    assert "tmem_alloc(" not in body[:body.index("pdl_wait();")]


def test_the_decode_step_s_early_start_waits():
    """Its attention waits in the producer warp, behind the tiles it loads early:
    a CTA without work has none, and waits before it returns."""
    body = dict(kernels(source("flash_decode.cu")))["flash_decode_splitk_kernel"]
    bad, _ = unwaited_returns(body)
    assert not bad, f"flash_decode_splitk_kernel returns without waiting for the kernel before it: {bad}"
    assert body.count("pdl_wait();") == 3  # at once without the early start; before a return; in the producer
