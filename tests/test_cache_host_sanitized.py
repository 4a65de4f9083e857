"""The host code of the rotary positions, the paged cache and its attention under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): their refusals, run as a child process against the sanitized build."""
import os
import subprocess
import sys

import pytest


def test_cache_host_suite_passes_under_asan_and_ubsan():
    import host_sanitize as H
    rt = H.runtimes()
    if rt is None:
        pytest.skip("g++ sanitizer runtimes are not installed")
    lib = H.build()
    env = dict(os.environ, LD_PRELOAD=":".join(rt), BSF8_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(H.ROOT, "tests", "test_cache_host.py")], cwd=H.ROOT, env=env, capture_output=True, text=True,
                       timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out
