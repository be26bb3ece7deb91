"""The sweep of appends with axes, cross attention and shared prefixes run by
test_gpu_kv8_more_debug_bounds.py in a child process against the bounds-checking
debug build (KVQ_LIB_PATH): every block size, head size, format and type, few
and many rows on either side, keys that CTA borders cut; every call must leave
the status word at 0 and match the oracle.  Not a test module itself."""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]

from test_gpu_kv8_more import TYPES, AxesRun, Groups, Run, cross  # noqa: E402
from bit_kv_cache_02_gb300 import kv8, kvq  # noqa: E402


def main():
    assert kvq.LIB_PATH == os.environ["KVQ_LIB_PATH"], "not the debug build"
    n = 0
    shapes = ((128, 32, 4), (64, 64, 7), (128, 128, 3), (64, 32, 2), (128, 64, 1), (64, 128, 1))
    for i, (fmt, dtype) in enumerate(TYPES):  # each block and head size with two of the types
        for D, B, g in shapes[i % 2::2]:
            r = AxesRun(kv8, 4, 2, g, D, B, fmt, dtype, 5 * B + 200, seed=B + g, rot=D // 2, interleaved=B == 64)
            for new in ([0, 1, B, 130], [B + 70, 129, 1, 3], [1, 1, 1, 1]):
                r.append(new)
                r.check_state()
            cross(r, [1, 3, 0, 2])
            cross(r, [100, 1, 30, 7])
            r = Groups(kv8, [3, 1, 4], [2 * B + 5, B, 3 * B], 2, g, D, B, fmt, dtype, 6 * B + 200, before=1, behind=1,
                       seed=B)
            for new in ([5, B, 1, 0, 40, 1, 2, 3, 7, 9], [1] * 10, [3, 70, 1, 2, 0, 20, 1, 1, 5, 1]):
                r.append(new)
                r.shared()
            n += 8
    for S, g, prefix in ((40, 8, 2500), (3, 2, 6000)):  # parts of long lines
        r = Groups(kv8, [S], [prefix], 2, g, 128, 64, "int8", "bfloat16", prefix + 300, seed=S)
        r.append([(5 * s) % 130 for s in range(S)])
        r.shared()
        r = Run(kv8, 2, 2, g, 64, 64, "e4m3", "float16", prefix + 100, seed=S)
        r.append([prefix, 30])
        cross(r, [S, 1])
        n += 2
    r = AxesRun(kv8, 3, 11, 1, 64, 32, "int8", "float16", 2300, seed=5, top=2300)  # eight heads at a time
    r.append([2200, 2100, 1900])
    r.check_state()
    print(f"bounds sweep ok: {n + 1} steps, {kvq.launch_count()} kernels")


if __name__ == "__main__":
    main()
