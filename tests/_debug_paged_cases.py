"""Small valid cases of the paged calls against whichever build of the library YOCO_LIB_PATH
names (the debug-checks build, from tests/test_gpu_paged_debug.py): results within their
bounds and no failed index check.  Prints "debug cases ok"."""
import ctypes
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import gated_retention_shared_gb300 as Y  # noqa: E402
import test_gpu_paged as T  # noqa: E402


def passed(name):
    w = ctypes.c_uint32(0xFFFFFFFF)
    assert Y.lib.yoco_debug_checks(1, ctypes.byref(w)) == Y.YOCO_OK, Y.lib.yoco_last_error()
    assert w.value == 0, (name, hex(w.value))


def main():
    assert os.environ.get("YOCO_LIB_PATH"), "run with YOCO_LIB_PATH set to the debug build"
    for dtype, d in T.TYPES:
        T.run_decode(Y, [0, 1, 127, 128, 700, 3000], 6, 2, d, 16, dtype)
        T.run_decode(Y, [900, 40], 6, 2, d, 64, dtype, window=300, sinks=4)
        passed(f"decode {dtype} {d}")
        T.run_prefill(Y, [1, 0, 70, 130], [0, 9, 500, 3], 6, 2, d, 16, dtype)
        T.run_prefill(Y, [5], [9000], 6, 2, d, 64, dtype)  # cut into pieces
        passed(f"prefill {dtype} {d}")
        T.test_append(Y, [3, 0, 40, 1], [0, 7, 29, 100], 4, 2, d, 16, dtype, 1e4, "dense")
        passed(f"append {dtype} {d}")
    print("debug cases ok")


if __name__ == "__main__":
    main()
