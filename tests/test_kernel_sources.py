"""The sources whose hash keeps the GEMM's counter summaries current are all that its
kernel is compiled from."""

import os
import re

import bench

CSRC = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "moe_grouped_gemm_02_amd", "csrc")


def test_kernel_sources_are_the_gemms_and_every_header_it_includes():
    seen, todo = set(), ["dg_gemm.hip"]
    while todo:
        name = todo.pop()
        if name in seen:
            continue
        seen.add(name)
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            names = re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M)
        todo += [n for n in names if os.path.exists(os.path.join(CSRC, n))]  # include/ holds declarations only
    assert set(bench.KERNEL_SOURCES) == seen and len(bench.KERNEL_SOURCES) == len(seen)
