"""The sizes of tests/test_gpu_paged_sizes.py, at which the paged-cache kernels
loop over heads and pages, against the bounds-checked debug build of the library
(RF_GB300_LIB=debug): each must leave the device status RF_OK and match the
oracle.  Run as a script by tests/test_gpu_paged_sizes_bounds.py, in a process of
its own; prints one line per case."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tests import test_gpu_paged_sizes as S  # noqa: E402


def main():
    import cascaded_reductions_loop_gb300 as rf
    assert rf.LIB_PATH.endswith("_dbg.so"), f"not the debug build: {rf.LIB_PATH}"

    def run(f, *args):
        f(rf, *args)
        st = rf.rf_get_device_status()
        assert st == rf.RF_OK, f"{f.__name__}{args}: device status {rf.rf_status_string(st)}"
        print(f"ok  {f.__name__} {args}", flush=True)

    for dtype in (S.BF16, S.F32):
        for d, rot, inter, norm in [(128, 128, False, True), (64, 32, True, True)]:
            run(S.test_qk_norm_rope_several_heads_a_lane_group, dtype, d, rot, inter, norm, 4, 9, 3)
        run(S.test_qk_norm_rope_tokens_far_apart, dtype)
    for case in [(128, 4, 5, 6, 64, (128, False, True)), (64, 8, 7, 7, 128, (64, True, True))]:
        run(S.test_bf16_append_several_heads_a_lane_group, *case)
    for ps, d, Hkv, rope in [(16, 64, 5, (64, False, True)), (16, 128, 7, (128, False, True)),
                             (64, 64, 7, (64, False, True)), (64, 128, 3, (128, True, True)),
                             (128, 128, 3, (128, False, True))]:
        for Hq in (0, 6):
            run(S.test_e4m3_prompts_several_pages_and_heads_a_cta, ps, d, Hkv, rope, Hq)
    for kind in ("e4m3", "bf16"):
        for new in (1, 5, 300):
            run(S.test_pages_beyond_32_bits, kind, new)
    print("bounds-checked build: every case of these sizes clean", flush=True)


if __name__ == "__main__":
    main()
