"""The selective-scan, short-convolution and draft-acceptance C-ABI tests
(tests/test_abi_scan.py) against the host-sanitized build of the library, as
test_abi_sanitized runs the others: built by

    python -m gated_delta_rule_79_amd.build --sanitize

and skipped without it."""

import os
import subprocess
import sys

import pytest

from gated_delta_rule_79_amd import build
from test_abi_sanitized import ROOT, _asan_runtime, _stale


def test_scan_abi_under_sanitizers():
    if not os.path.exists(build.ASAN_LIB) or _stale(build.ASAN_LIB):
        pytest.skip("host-sanitized library not built from these sources (build.py --sanitize)")
    rt = _asan_runtime()
    if rt is None:
        pytest.skip("AddressSanitizer runtime not found")
    env = dict(os.environ, LD_PRELOAD=rt, GDN_LIBRARY=build.ASAN_LIB,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_scan.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out
