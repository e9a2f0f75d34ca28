"""The host code of the transformer block's entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU): a child process with the sanitizer runtime
drives them through their argument checks and launch preparation."""

import os
import re
import subprocess
import sys

import pytest

from tests.test_host_sanitizers import ASAN_LIB, ROOT, _runtime

HEADER = os.path.join(ROOT, "include", "dg_block.h")
DRIVER = os.path.join(ROOT, "tests", "block_host_sanitizer_driver.py")


@pytest.mark.skipif(not os.path.exists(ASAN_LIB), reason="libdg_host_asan.so not built (build.py)")
def test_block_entry_points_under_host_sanitizers():
    env = dict(os.environ)
    env["LD_PRELOAD"] = _runtime() + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    env["HIP_VISIBLE_DEVICES"] = "-1"  # the launches must fail: the addresses are fake
    env["DG_NUM_CUS"] = "256"  # the GEMMs' work division asks for it
    res = subprocess.run([sys.executable, DRIVER, ASAN_LIB, HEADER], env=env, capture_output=True, text=True, timeout=600)
    reports = [line for line in res.stderr.splitlines() if "Sanitizer" in line or "runtime error" in line]
    assert res.returncode == 0 and not reports, res.stdout[-2000:] + "\n" + res.stderr[-6000:]
    m = re.fullmatch(r"block host-sanitizer driver ok calls=(\d+) entries=(\d+)", res.stdout.strip().splitlines()[-1])
    assert m and int(m.group(1)) > 5000 and int(m.group(2)) == 13
