"""The decode-step boundary tests again, against the library's host code built with
AddressSanitizer and UndefinedBehaviorSanitizer.  Nothing here launches a kernel."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_step_boundary_tests_pass_under_asan_and_ubsan():
    from gemv_prefill_decode_amd import build as b
    objects = [os.path.join(b.BUILD_DIR, s + ".o") for s in b.SOURCES]
    if not all(os.path.exists(o) for o in objects):
        pytest.skip("regular build objects missing (run __graft_entry__.build())")
    try:
        fresh = os.path.exists(b.SAN_OUT) and os.path.getmtime(b.SAN_OUT) > max(map(os.path.getmtime, objects))
        san = b.SAN_OUT if fresh else b.build_sanitized()
        rt = b.asan_runtime()
    except (RuntimeError, FileNotFoundError) as e:
        pytest.skip(f"no sanitizer toolchain: {e}")
    env = dict(os.environ, QMM_LIBRARY=san, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join("tests", "test_step_boundary.py"), "-q",
                        "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, out
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr, out
