"""A kernel that may begin while its stream's previous one still runs does not read by the path for data that nothing writes
during the kernel: what it reads may be that kernel's output."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "top_sampling_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__restrict__|LDG\.CONSTANT")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_no_read_only_loads_in_overlapped_kernels():
    files = {f: _code(f) for f in os.listdir(CSRC)}
    overlapped = {f for f, s in files.items() if re.search(r"^\s*begin_overlapped\(\);", s, re.M)}
    assert {"vsamp_block_matmul.cuh", "vsamp_block_quant.cuh", "vsamp_adamw.cuh", "vsamp_score.cuh"} <= overlapped
    # and the device code that they include
    reach = set(overlapped)
    while True:
        more = {h for f in reach for h in re.findall(r'#include "(\w+\.cuh)"', files[f])} - reach
        if not more:
            break
        reach |= more
    found = {f: READ_ONLY.findall(files[f]) for f in sorted(reach) if READ_ONLY.search(files[f])}
    assert not found, found
