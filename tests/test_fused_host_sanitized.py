"""The host code of the operators around the products under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only):
their refusals, handles and describe lines, run as a child process against the sanitized build."""
import os
import subprocess
import sys

import pytest


def test_fused_host_suites_pass_under_asan_and_ubsan():
    import host_sanitize as H
    rt = H.runtimes()
    if rt is None:
        pytest.skip("g++ sanitizer runtimes are not installed")
    lib = H.build()
    nm = subprocess.run(["nm", os.path.join(H.OUT, "bsf8_host.o")], capture_output=True, text=True).stdout
    assert "__asan_report" in nm and "__ubsan_handle" in nm, "the host object is not instrumented"
    env = dict(os.environ, LD_PRELOAD=":".join(rt), BSF8_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    suites = [os.path.join(H.ROOT, "tests", f) for f in ("test_fused_host.py", "test_fused_describe.py", "test_far_rows_host.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu"] + suites,
                       cwd=H.ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out
