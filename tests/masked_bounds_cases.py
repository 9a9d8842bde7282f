"""Masked attention against the bounds-checked debug build of the library
(librf_gb300_dbg.so, selected by RF_GB300_LIB=debug): cases of each entry point must
leave the device status RF_OK and match the oracle.  Run as a script by
tests/test_gpu_masked_bounds.py, in a process of its own; prints one line per case."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tests import test_gpu_masked as M  # noqa: E402
from tests import test_gpu_window as W  # noqa: E402


def main():
    import cascaded_reductions_loop_gb300 as rf
    assert rf.LIB_PATH.endswith("_dbg.so"), f"not the debug build: {rf.LIB_PATH}"

    def ok(what):
        st = rf.rf_get_device_status()
        assert st == rf.RF_OK, f"{what}: device status {rf.rf_status_string(st)}"
        print(f"ok  {what}", flush=True)

    for case in range(len(M.WINDOWS)):
        if sum(M.WINDOWS[case][8]) < 30000:
            M.test_window(rf, case)
            ok(f"window {M.WINDOWS[case][:8]}")
    for case in range(len(M.TREES)):
        M.test_tree(rf, case)
        ok(f"tree {M.TREES[case][:9]}")
    for kind, Tq, Hq, tree in M.ODD_VALUES:
        M.test_values_that_are_not_finite_reach_only_the_rows_that_read_them(rf, kind, Tq, Hq, tree)
        ok(f"values that are not finite {kind} {Tq} x {Hq}")
    for case in range(len(W.CASES)):
        W.test_prompts(rf, case)
        ok(f"prompts {W.CASES[case][:5]}")
    for which in ("k", "v"):
        for d, Hq in ((64, 1), (128, 4)):
            W.test_values_that_are_not_finite_reach_only_the_rows_that_read_them(rf, which, d, Hq)
            ok(f"prompts with {which} that are not finite, d {d}")
    W.test_views_of_a_fused_projection_and_rows_left_alone(rf)
    ok("views of a fused projection")
    print("bounds-checked build: every masked case clean", flush=True)


if __name__ == "__main__":
    main()
