"""Masked attention on the GPU where the kernel's warps wait for one another in an order
that not every piece of work has all of: query tiles that are missing, sequences that
read nothing.  Against the fp64 oracle, and again and again with the same bits.

Tolerances as in tests/test_gpu_masked_values.py."""
import numpy as np
import pytest
import torch

from tests import test_gpu_window as W
from tests.helpers import to64
from tests.test_gpu_masked import masked_reference, rf, run, tree_of  # noqa: F401
from tests.test_gpu_masked_values import MANY
from tests.test_gpu_paged import BF16, Batch, _gen

pytestmark = pytest.mark.gpu


def again_and_again(rf, bt, q, scale, what, window=0, sinks=0, parents=None, calls=25):  # noqa: F811
    """The oracle's result, and the same bits in every call, with L2 full of other data or not."""
    got, status = run(rf, bt, q, scale, window, sinks, parents)
    assert status == rf.RF_OK, what
    ref, tol = masked_reference(q, bt, scale, window, sinks, parents, **MANY)
    err = np.abs(to64(got) - ref)
    assert (err <= tol).all(), f"{what}: worst {np.nanmax(err / tol):.2f} of the tolerance"
    cache, qd = bt.device(rf), q.cuda()
    B, Tq, Hq, d = q.shape
    ws = torch.empty(rf.rf_attn_decode_paged_ex_workspace_size(B, Hq, bt.Hkv, Tq, d), dtype=torch.uint8,
                     device="cuda")
    mask = rf.rf_attn_mask(window, sinks, None if parents is None else
                           torch.tensor(parents, dtype=torch.int32).cuda())
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(calls):
        if i % 2:
            other.fill_(i)
        o = torch.full_like(qd, 7.0)
        rf.rf_attn_decode_paged_ex(cache, qd, o, scale, mask, ws)
        assert torch.equal(o, got), f"{what}: call {i} gives other bits"
    assert rf.rf_get_device_status() == rf.RF_OK


LAST_ALONE = [
    # kind, d, Hkv, group, query tokens, tree, window, sinks, lens
    ("e4m3", 128, 4, 8, 40, True, 0, 0, [40 + 37 * i % 260 for i in range(12)]),
    ("e4m3", 128, 4, 8, 40, False, 90, 4, [40 + 53 * i % 900 for i in range(40)]),
    ("e4m3", 128, 2, 8, 33, True, 0, 0, [33, 3000, 300, 60, 9000, 170, 40, 41]),
    ("e4m3", 128, 2, 5, 60, True, 0, 0, [60 + 91 * i % 700 for i in range(50)]),
    ("e4m3", 64, 2, 8, 40, True, 0, 0, [40 + 37 * i % 500 for i in range(50)]),
    ("e4m3", 64, 1, 5, 60, False, 200, 3, [60, 5000, 90, 1200] * 4),
    ("bf16", 128, 4, 8, 40, True, 0, 0, [40 + 53 * i % 700 for i in range(24)]),
    ("bf16", 64, 2, 5, 60, False, 64, 3, [60 + 91 * i % 900 for i in range(50)]),
]


@pytest.mark.parametrize("case", range(len(LAST_ALONE)))
def test_last_pairs_of_one_tile(rf, case):  # noqa: F811
    kind, d, Hkv, G_, Tq, tree, window, sinks, lens = LAST_ALONE[case]
    assert 0 < Tq % (2 * (128 // G_)) <= 128 // G_
    bt = Batch(kind, lens, Hkv, d, 64, seed=1100 + case).garbage()
    q = torch.randn(len(lens), Tq, Hkv * G_, d, generator=_gen(1120 + case)).to(BF16)
    parents = [tree_of(_gen(1140 + b), Tq) for b in range(len(lens))] if tree else None
    again_and_again(rf, bt, q, d ** -0.5, LAST_ALONE[case][:8], window, sinks, parents)


NO_KEYS = [
    # d, Hq, Hkv, window, sinks, new tokens, keys: prompts of one and two query tiles, some
    # of which read nothing, several to a CTA
    (128, 4, 1, 16, 2, [300, 1, 30, 33, 40, 300], [0, 1, 0, 10, 0, 300]),
    (64, 8, 8, 0, 0, [300, 1, 128, 129, 40, 300, 77] * 6, [0, 1, 0, 10, 0, 300, 500] * 6),
    (128, 32, 8, 100, 4, [32, 64, 1, 70, 32, 0, 60, 33] * 6, [0, 0, 0, 90, 0, 0, 0, 300] * 6),
    (128, 40, 8, 0, 0, [51, 20, 1, 25, 26] * 9, [0, 0, 3, 0, 400] * 9),
    (64, 16, 16, 200, 130, [400, 128, 128, 1, 500], [250, 0, 0, 0, 3]),
]


@pytest.mark.parametrize("case", range(len(NO_KEYS)))
def test_prompts_whose_rows_read_nothing(rf, case):  # noqa: F811
    d, Hq, Hkv, window, sinks, new, keys = NO_KEYS[case]
    q, k, v = W.inputs(new, keys, Hq, Hkv, d, 1200 + case)
    ref, tol = W.reference(q, k, v, new, keys, d ** -0.5, window, sinks)
    q, k, v, cq, ck = (t.cuda() for t in (q, k, v, W._cu(new), W._cu(keys)))
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(25):
        if i % 2:
            other.fill_(i)
        o = torch.full_like(q, 7.0)
        rf.rf_attn_fwd_window(q, k, v, o, d ** -0.5, window, sinks, cq, ck, max(new))
        if first is None:
            W.assert_close(o, ref, tol, NO_KEYS[case])
            first = o
        assert torch.equal(o, first), f"call {i} gives other bits"
        a = q.clone()                                  # in place
        rf.rf_attn_fwd_window(a, k, v, a, d ** -0.5, window, sinks, cq, ck, max(new))
        assert torch.equal(a, first), f"call {i} in place gives other bits"
    assert rf.rf_get_device_status() == rf.RF_OK


def empties(n, of, times):
    """n sequences without tokens in front of each of the others."""
    return ([x for i in of for x in [0] * n + [i]]) * times


EMPTIES = [
    # kind, d, Hkv, group, query tokens, tree, window, sinks, lens: what lies behind a
    # sequence's last token in its last page is not finite
    ("bf16", 128, 4, 4, 16, True, 0, 0, empties(3, [37, 20, 300], 24)),
    ("bf16", 128, 2, 8, 40, True, 0, 0, empties(2, [41, 700], 30)),
    ("bf16", 64, 4, 4, 16, False, 50, 3, empties(5, [17, 130, 40], 16)),
    ("bf16", 128, 1, 4, 40, False, 60, 0, [5, 1, 39, 70, 3, 0, 2, 200] * 24),
    ("e4m3", 128, 4, 4, 16, True, 0, 0, empties(3, [37, 20, 300], 24)),
    ("e4m3", 128, 2, 8, 40, True, 0, 0, empties(2, [41, 700], 30)),
    ("e4m3", 64, 4, 8, 16, False, 50, 3, empties(5, [17, 130, 40], 16)),
    ("e4m3", 128, 1, 4, 40, False, 60, 0, [5, 1, 39, 70, 3, 0, 2, 200] * 24),
]


@pytest.mark.parametrize("case", range(len(EMPTIES)))
def test_sequences_that_read_nothing_in_front_of_unread_nans(rf, case):  # noqa: F811
    kind, d, Hkv, G_, Tq, tree, window, sinks, lens = EMPTIES[case]
    bt = Batch(kind, lens, Hkv, d, 64, seed=1300 + case).garbage()
    q = torch.randn(len(lens), Tq, Hkv * G_, d, generator=_gen(1320 + case)).to(BF16)
    parents = [tree_of(_gen(1340 + b), Tq) for b in range(len(lens))] if tree else None
    again_and_again(rf, bt, q, d ** -0.5, EMPTIES[case][:8], window, sinks, parents)


def test_prompts_that_read_nothing_in_front_of_unread_nans(rf):  # noqa: F811
    """Infinities and NaN in values that no row reads: of the next sequence, behind a
    prompt's last key in its last key tile, and between the sinks and the window."""
    new, keys = [300, 33, 32, 32, 40, 7] * 8, [10, 0, 0, 5, 140, 60] * 8
    window, sinks, scale = 30, 4, 128 ** -0.5
    q, k, v = W.inputs(new, keys, 8, 2, 128, 1400)
    ref, tol = W.reference(q, k, v, new, keys, scale, window, sinks)
    at = 0
    for i, (n, nk) in enumerate(zip(new, keys)):
        if nk == 60:
            v[at + sinks:at + nk - n + 1 - window] = float("nan") if i % 4 == 1 else float("inf")
        at += nk
    assert not torch.isfinite(v).all()
    q, k, v, cq, ck = (t.cuda() for t in (q, k, v, W._cu(new), W._cu(keys)))
    first = None
    for i in range(25):
        o = torch.full_like(q, 7.0)
        rf.rf_attn_fwd_window(q, k, v, o, scale, window, sinks, cq, ck, max(new))
        if first is None:
            W.assert_close(o, ref, tol, "unread")
            first = o
        assert torch.equal(o, first), f"call {i} gives other bits"
    assert rf.rf_get_device_status() == rf.RF_OK


SKIPPED = [
    # kind, d, Hkv, group, query tokens, window, sinks, lens: key tiles that one of a pair's
    # query tiles takes and the other does not, at either end and behind the sinks
    ("e4m3", 64, 2, 1, 256, 128, 0, [256 + 331 * i % 3000 for i in range(12)]),
    ("e4m3", 64, 2, 2, 130, 1, 300, [130 + 331 * i % 3000 for i in range(24)]),
    ("e4m3", 128, 2, 1, 256, 200, 1, [256 + 331 * i % 2000 for i in range(12)]),
    ("bf16", 64, 2, 1, 256, 128, 130, [256 + 331 * i % 3000 for i in range(12)]),
    ("bf16", 128, 1, 2, 128, 64, 0, [128 + 331 * i % 2000 for i in range(24)]),
]


@pytest.mark.parametrize("case", range(len(SKIPPED)))
def test_key_tiles_that_one_of_two_query_tiles_takes(rf, case):  # noqa: F811
    kind, d, Hkv, G_, Tq, window, sinks, lens = SKIPPED[case]
    bt = Batch(kind, lens, Hkv, d, 32, seed=1500 + case).garbage()
    q = torch.randn(len(lens), Tq, Hkv * G_, d, generator=_gen(1520 + case)).to(BF16)
    again_and_again(rf, bt, q, d ** -0.5, SKIPPED[case][:7], window, sinks)
