"""Host memory that runs out inside a call comes back as a status: no C++
exception leaves a C entry point."""
import os
import subprocess
import sys

import kv_cached_gqa_rope_gb300 as kv

CHILD = """
import resource
import kv_cached_gqa_rope_gb300 as kv
with open("/proc/self/statm") as f:
    used = int(f.read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (256 << 20), used + (256 << 20)))
try:
    kv.SlotTable(2 ** 31 - 1, 8)
except kv.KvgqaError as e:
    print("code", e.code)
t = kv.SlotTable(4, 8)
print("row", t.admit(1, 3))
"""


def test_a_table_too_large_for_the_host():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["code", "ENOMEM", "row", "0"]


def test_the_status_has_its_name():
    assert kv.STATUS_NAMES[10] == "ENOMEM"
