"""The 8-bit chunk cache's host code (argument checks, the choice of a call's form, workspace
offsets, launch set-up) under AddressSanitizer and UndefinedBehaviorSanitizer: its host-side ABI
tests in a child process against a library whose host sources are built sanitized (no GPU needed)."""
import os
import subprocess
import sys

import pytest

from test_abi_sanitized import ROOT, _asan_runtime


def test_cache8_host_code_sanitized(tmp_path):
    rt = _asan_runtime()
    if rt is None:
        pytest.skip("no shared ASan runtime in this toolchain")
    from gated_deltanet_hybrid_amd import build
    objs = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES
            if s not in build.HOST_SOURCES]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library's objects are not built")
    lib = build.build_host_sanitized(str(tmp_path / "libhla_san.so"))
    env = dict(os.environ, HLA_LIBRARY=lib, LD_PRELOAD=rt, PYTHONPATH=ROOT,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_abi_cache8_cpu.py"), "-q",
                        "-p", "no:cacheprovider"], env=env, capture_output=True, text=True, timeout=600,
                       cwd=str(tmp_path))
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
