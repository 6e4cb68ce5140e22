"""The cache calls in the debug build (every plain global load and store checked
against its tensor's extent): the parity tests of test_cache_ops_gpu.py, which
read the device status after every call, run against libgbattn_debug.so.  The
library is chosen per process, so they run in a child."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_index_check_fires():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_flashattention_fwd_gb300 import build

    build.build()
    build.build(debug=True)
    run = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", "not inf and not 32_bits",
         os.path.join(ROOT, "tests", "test_cache_ops_gpu.py")],
        cwd=ROOT, env=dict(os.environ, GBATTN_DEBUG="1"), capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stdout[-3000:] + run.stderr[-1000:]
