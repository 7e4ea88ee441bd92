"""The host code of the serving entry points (4-bit weights, 8-bit cache) under
AddressSanitizer and UndefinedBehaviorSanitizer: their ABI test modules run
against the library built as in test_host_sanitizers.  No GPU is used."""

import os
import subprocess
import sys

from fp8_block_scaled_nt_amd import build as B
from tests.test_host_sanitizers import sanitized_lib  # noqa: F401

MODULES = ["test_abi_serving.py", "test_abi_serving_empty.py", "test_abi_forced_ways.py"]


def test_serving_abi_clean_under_sanitizers(sanitized_lib):  # noqa: F811
    lib, runtime = sanitized_lib
    env = dict(os.environ)
    env.update({"DG_LIBRARY": lib, "LD_PRELOAD": runtime,
                "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1:abort_on_error=0",
                "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"})
    r = subprocess.run([sys.executable, "-m", "pytest", *(os.path.join(B.ROOT, "tests", m) for m in MODULES), "-q",
                        "-p", "no:cacheprovider"], cwd=B.ROOT, env=env, capture_output=True, text=True, timeout=600)
    text = r.stdout + r.stderr
    assert r.returncode == 0, text[-4000:]
    assert "AddressSanitizer" not in text and "runtime error" not in text, text[-4000:]
    assert " passed" in text
