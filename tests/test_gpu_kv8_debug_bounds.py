"""The 8-bit cache under the bounds-checking debug build (compiled with
KVQ_DEBUG_BOUNDS): indices that the kernels compute on the device into the
cache, the row tensors, the rotation table and the workspace are checked, and
one out of range would set KVQ_STATUS_BOUNDS.  _bounds_sweep_kv8.py runs against
that build in a child process."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sweep_under_the_debug_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_kv_cache_02_gb300 import build
    lib = build.build_debug()
    env = dict(os.environ, KVQ_LIB_PATH=lib)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_bounds_sweep_kv8.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "bounds sweep ok" in r.stdout
