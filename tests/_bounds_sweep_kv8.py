"""The 8-bit cache's sweep run by test_gpu_kv8_debug_bounds.py in a child
process against the bounds-checking debug build (KVQ_LIB_PATH): prompts,
chunks, drafts and single tokens for every block size, head size, format and
type, row ranges that do not begin at row 0, items that CTA borders cut, long
appends whose CTAs take several heads; every call must leave the status word
at 0 and match the oracle.  Not a test module itself."""

import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]

from test_gpu_kv8 import Run, TYPES  # noqa: E402
from bit_kv_cache_02_gb300 import kv8, kvq  # noqa: E402


def step(r, new, **kw):
    r.append(new)
    r.check_state()
    r.attend(**kw)
    assert int(r.cache.status.item()) == 0


def main():
    assert kvq.LIB_PATH == os.environ["KVQ_LIB_PATH"], "not the debug build"
    n = 0
    for fmt, dtype in TYPES:
        for D, B, g in ((128, 32, 4), (128, 64, 1), (128, 128, 3), (64, 32, 2), (64, 64, 7), (64, 128, 1)):
            r = Run(kv8, 4, 2, g, D, B, fmt, dtype, 5 * B + 200, seed=B + g, rot=D // 2, interleaved=B == 64)
            for new in ([0, 1, B, 130], [B + 70, 129, 1, 3], [2, 8, 5, 1], [1, 1, 1, 1]):
                step(r, new)
                n += 1
    for new in ([3, 1], [120, 1], [1, 90]):  # parts of long lines
        r = Run(kv8, 2, 2, 2, 128, 64, "int8", "bfloat16", 6000, seed=4)
        r.append([5000, 300])
        step(r, new)
        n += 1
    r = Run(kv8, 3, 11, 1, 64, 32, "int8", "float16", 9000, seed=5)  # keys and values apart, eight heads at a time
    r.append([8600, 8000, 8200])
    r.check_state()
    r.append(np.array([1, 1, 1]).tolist())
    r.attend()
    assert int(r.cache.status.item()) == 0
    print(f"bounds sweep ok: {n + 1} steps, {kvq.launch_count()} kernels")


if __name__ == "__main__":
    main()
