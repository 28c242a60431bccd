"""The argument checks of linear attention and the layer norm under AddressSanitizer and
UndefinedBehaviorSanitizer (host code, CPU): tests/test_attn_abi.py against a library built as for the
recurrences' checks."""
import os
import subprocess
import sys

import pytest

from linear_rnn_sequence_wkv7_amd import build as B
from tests.test_host_sanitizers import CHILD, ROOT


@pytest.mark.timeout(900)
def test_attn_abi_under_host_sanitizers(tmp_path):
    try:
        runtime = B.sanitizer_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    if runtime is None:
        pytest.skip("no clang sanitizer runtime in the toolchain")
    lib = B.build_host_sanitized(str(tmp_path / "hostsan"))
    env = {**os.environ, "LD_PRELOAD": runtime, "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1",
           "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"}
    child = CHILD.replace("tests/test_abi.py", "tests/test_attn_abi.py").format(root=ROOT, lib=lib)
    r = subprocess.run([sys.executable, "-c", child], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "passed" in r.stdout and "failed" not in r.stdout, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
