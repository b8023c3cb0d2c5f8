"""The token mixers' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): their
refusal tests run in a child process against the library's sanitized host build."""
import os
import subprocess
import sys

import pytest

from tests.test_sanitized_host import ROOT, _runtime


def test_mixers_host_code_is_clean_under_sanitizers(tmp_path):
    from chunked_gated_delta_13_amd import build as kbuild
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not asan or not ubsan:
        pytest.skip("gcc sanitizer runtimes not installed")
    if not (os.path.isdir(kbuild.BUILD_DIR) and any(f.endswith(".hip.o") for f in os.listdir(kbuild.BUILD_DIR))):
        pytest.skip("no device objects: the regular build has not run here")
    lib = kbuild.build_sanitized(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=f"{asan} {ubsan}",
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-p", "no:cacheprovider",
                        f"--kda-library={lib}", "tests/test_mixers_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-3000:]
    print(tail)
    assert r.returncode == 0, tail
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr, tail
