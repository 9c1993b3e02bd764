"""The C ABI checks of tests/test_feedforward_abi.py against the host-sanitized
build of the API layer (see test_sanitized_abi.py)."""
import os
import subprocess
import sys

import pytest

from exact_range_similarity_amd import build as ersj_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_feedforward_abi_checks_pass_under_sanitizers():
    try:
        rt = ersj_build.sanitizer_runtime()
    except FileNotFoundError as e:
        pytest.skip(str(e))
    lib = ersj_build.build_sanitized()
    env = dict(os.environ)
    env.update(ERSJ_LIBRARY=lib, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_feedforward_abi.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert " passed" in r.stdout
