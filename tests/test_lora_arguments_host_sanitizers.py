"""The adapters' checks of their arguments under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only; every call of that suite returns
before the first HIP call)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checks_of_arguments_under_host_sanitizers():
    from quantized_matmul_qgemv_amd import build as B
    try:
        lib = B.build_host_sanitized()
        rt = B.asan_runtime()
    except (RuntimeError, FileNotFoundError) as e:
        pytest.skip(f"no sanitizer toolchain: {e}")
    env = dict(os.environ, QMM_LIBRARY=lib, LD_PRELOAD=rt, HIP_VISIBLE_DEVICES="",
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0:exitcode=86",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=87")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_lora_arguments_cpu.py"),
                        "-x", "-q", "-s", "-p", "no:cacheprovider", "-m", "not gpu"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-6000:]
    assert " passed" in out, out[-3000:]
