"""Small valid cases of the scored paged calls, the scaled rotary calls and the page calls against
whichever build of the library YOCO_LIB_PATH names (the debug-checks build, from
tests/test_gpu_paged_more_debug.py): results within their bounds and no failed index check.  Prints
"debug cases ok"."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import gated_retention_shared_gb300 as Y  # noqa: E402
import test_gpu_paged_pool as Pool  # noqa: E402
import test_gpu_paged_round as Round  # noqa: E402
import test_gpu_paged_scored as S  # noqa: E402
import test_gpu_rope_scaled as R  # noqa: E402
from _debug_paged_cases import passed  # noqa: E402


def main():
    assert os.environ.get("YOCO_LIB_PATH"), "run with YOCO_LIB_PATH set to the debug build"
    for dtype, d in S.TYPES:
        for name in ("all", "window all", "low cap"):
            S.test_decode(Y, dtype, d, name)
            S.test_prefill(Y, dtype, d, name)
        S.test_prefill_cut_into_pieces(Y, dtype, d, "docs tail")
        passed(f"scored {dtype} {d}")
    for layout in ("pairs", "halves"):
        R.test_rows_at_positions(Y, "bf16", 128, 48, layout, {})
        R.test_sizes_in_place_and_strided(Y, "f32", layout, 700, 3)
        R.test_append(Y, "bf16", 128, dict(layout=layout, rotary_dim=32))
        passed(f"rope {layout}")
    Pool.test_random_rounds(Y, 60, 300, 32, 30, 1, 128, Pool.torch.bfloat16, 1)
    Pool.test_a_call_without_room_changes_nothing_but_what_shrinks(Y)
    Round.test_serving_rounds(Y, "bf16", 128, 6, 2, 16, False)
    passed("pages")
    print("debug cases ok")


if __name__ == "__main__":
    main()
