"""The values and streamed suites of the image operators under the checked build
(every store, asynchronous copy and slot tested against its extent)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("memory_bound_normalization_gb300")
from memory_bound_normalization_gb300 import _lib  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_under_checks():
    from memory_bound_normalization_gb300 import build as libbuild

    if _lib.checked_variant():
        pytest.skip("runs the checked build already")
    libbuild.build(checked=True)
    env = dict(os.environ, RMSNORM_LIBRARY_VARIANT="checked")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_group_norm_values_gpu.py", "tests/test_group_norm_streamed_gpu.py",
           "tests/test_rope_values_gpu.py", "tests/test_image_modules_gpu.py"]
    out = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = (out.stdout + out.stderr)[-4000:]
    assert out.returncode == 0, tail
    assert " passed" in tail and " failed" not in tail, tail
