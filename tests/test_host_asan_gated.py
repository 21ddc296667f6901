"""The gated block's and the adapter pools' entry points' argument validation under host
AddressSanitizer (CPU only): tests/host_asan_gated.c against the library of
tests/test_host_asan.py, whose host code is instrumented."""

import os
import subprocess

import pytest

# (left out, as this file is, where only the GPU tests are wanted)
host_asan = pytest.importorskip("tests.test_host_asan")
OUT, ROOT, _clang, _run = host_asan.OUT, host_asan.ROOT, host_asan._clang, host_asan._run
driver = host_asan.driver   # the fixture that builds the library


def test_gated_validation_is_clean_under_asan(driver):
    exe = os.path.join(OUT, "host_asan_gated")
    _run([_clang(), "-fsanitize=address", "-fno-omit-frame-pointer", "-g", "-O1",
          "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "host_asan_gated.c"),
          "-o", exe, "-L", OUT, "-lqlora_asan", f"-Wl,-rpath,{OUT}"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "host asan gated OK" in r.stdout, r.stdout + r.stderr
    assert "AddressSanitizer" not in r.stderr, r.stderr
