"""The paged-cache operators against the bounds-checked debug build of the
library (librf_gb300_dbg.so, selected by RF_GB300_LIB=debug): ragged cases of
each must leave the device status RF_OK and match the oracle.  Run as a script
by tests/test_gpu_paged_bounds.py, in a process of its own; prints one line per
case."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tests import test_gpu_paged as T  # noqa: E402
from tests.helpers import Guarded  # noqa: E402


def main():
    import cascaded_reductions_loop_gb300 as rf
    assert rf.LIB_PATH.endswith("_dbg.so"), f"not the debug build: {rf.LIB_PATH}"

    def ok(what):
        st = rf.rf_get_device_status()
        assert st == rf.RF_OK, f"{what}: device status {rf.rf_status_string(st)}"
        print(f"ok  {what}", flush=True)

    for dtype in (T.BF16, T.F32):
        for d, rot, inter, norm in [(128, 128, False, True), (64, 48, True, True), (64, 0, False, True)]:
            for n, Hq, Hkv in [(1, 1, 1), (67, 9, 3), (3000, 5, 2)]:
                nr = T.NR(rf, d, rot, inter, norm, dtype)
                x = torch.randn(n, Hq + Hkv, d, generator=T._gen(n)).to(dtype)
                pos = (torch.arange(n, dtype=torch.int32) * 7) % 600
                dev = x.cuda()
                qo, ko = Guarded((n, Hq, d), dtype), Guarded((n, Hkv, d), dtype)
                rf.rf_qk_norm_rope(dev[:, :Hq], dev[:, Hq:], qo.t, ko.t, nr.dev, pos.cuda())
                T.assert_rows(qo.t, nr.ref(x[:, :Hq], pos, "q"), dtype, "q")
                T.assert_rows(ko.t, nr.ref(x[:, Hq:], pos, "k"), dtype, "k")
                qo.check("q")
                ko.check("k")
                ok(f"norm and rotation {dtype} {n} x {Hq}+{Hkv} x {d}, rot {rot}")
    for case in range(len(T.APPENDS)):
        T.test_append(rf, case)
        ok(f"append {T.APPENDS[case][:4]}")
    for between, tokens in [(1, 100), (41, 2000)]:
        T.test_append_of_tokens_that_several_sequences_claim(rf, between, tokens)
        ok(f"append, {tokens} tokens claimed twice")
    for case in range(len(T.ATTNS)):
        if sum(T.ATTNS[case][6]) < 30000:
            T.test_attn_decode_paged(rf, case)
            ok(f"attention {T.ATTNS[case][:6]}")
    print("bounds-checked build: every paged case clean", flush=True)


if __name__ == "__main__":
    main()
