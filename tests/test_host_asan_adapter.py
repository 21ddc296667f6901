"""The dropout and 8-bit entry points' argument validation under host
AddressSanitizer (CPU only): tests/host_asan_adapter.c against the library of
tests/test_host_asan.py, whose host code is instrumented."""

import os
import subprocess

from tests.test_host_asan import OUT, ROOT, _clang, _run, driver  # noqa: F401  (driver: the fixture that builds it)


def test_adapter_validation_is_clean_under_asan(driver):  # noqa: F811
    exe = os.path.join(OUT, "host_asan_adapter")
    _run([_clang(), "-fsanitize=address", "-fno-omit-frame-pointer", "-g", "-O1",
          "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "host_asan_adapter.c"),
          "-o", exe, "-L", OUT, "-lqlora_asan", f"-Wl,-rpath,{OUT}"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "host asan adapter OK" in r.stdout, r.stdout + r.stderr
    assert "AddressSanitizer" not in r.stderr, r.stderr
