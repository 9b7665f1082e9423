"""The dense entry points' host code under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU, no GPU): their checks, the workspace sizes and the
choice of tile shapes run against liblq_san.so in a child process."""
import os
import subprocess
import sys

import pytest

from bit_ptq_looped_b200 import build as B
from test_sanitized_abi import ROOT, _runtime


def test_dense_checks_under_host_sanitizers():
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not (asan and ubsan):
        pytest.skip("gcc sanitizer runtimes not installed")
    B.build()  # or the child would start the compiler under the sanitizers
    env = dict(os.environ, LQ_LIB_PATH=B.build_sanitized(), LD_PRELOAD=f"{asan}:{ubsan}",
               ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    files = [os.path.join(ROOT, "tests", f) for f in ("test_dense_abi.py",
                                                      "test_dense_abi_limits.py")]
    # -s: a report of the sanitizer goes to this process, not into a captured test
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-q", "-s", "-p",
                        "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=900)
    log = r.stdout + r.stderr
    assert r.returncode == 0, log[-3000:]
    assert "AddressSanitizer" not in log and "runtime error:" not in log, log[-3000:]
