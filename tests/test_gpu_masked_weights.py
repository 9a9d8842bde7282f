"""Masked attention over a bf16 cache with heads of 64 and 17 to 32 query rows a kv head:
the header gives one rounding of the weights to bf16 from 33 rows on only, so these carry
two bf16 parts, 2^-16 of a weight.

Values are built so that each row's products nearly cancel: then the output's own rounding
(2^-8 of what is left) does not hide a lost low part.  Tolerances as in
tests/test_gpu_masked.py, with the border between one part and two at 32 rows."""
import numpy as np
import pytest
import torch

from oracle import paged as G
from tests import test_gpu_masked as M
from tests.helpers import to64
from tests.test_gpu_masked import masked_reference, rf, run, tree_of  # noqa: F401
from tests.test_gpu_paged import BF16, Batch, _gen


def softmax_rows(bt, q, scale, seen):
    """Weights [rows, n] of sequence 0's rows (query token, head) over its n keys."""
    n, Tq, Hq = bt.lens[0], q.shape[1], q.shape[2]
    at = bt.table[0].numpy()[np.arange(n) // bt.ps]
    k = to64(bt.pages[0])[at, 0, np.arange(n) % bt.ps]
    p = np.zeros((Tq * Hq, n))
    for t in range(Tq):
        s = scale * to64(q[0, t]) @ k[seen[t]].T
        e = np.exp(s - s.max(1, keepdims=True))
        p[t * Hq:(t + 1) * Hq, seen[t]] = e / e.sum(1, keepdims=True)
    return p


def cancelling(n, Tq, G_, window, sinks, tree, seed):
    """A batch of one sequence, its queries, parents and (rounded) weights; its values lie
    in the null space of the weights but for their own rounding to bf16."""
    bt = Batch("bf16", [n], 1, 64, 16, seed=seed, loud=0.0)
    q = torch.randn(1, Tq, G_, 64, generator=_gen(seed + 1)).to(BF16)
    parents = [tree_of(_gen(seed + 2), Tq)] if tree else None
    seen = [G.seen_keys(n, Tq, t, window, sinks, parents[0] if tree else None) for t in range(Tq)]
    p = softmax_rows(bt, q, 0.25, seen)
    null = np.linalg.svd(p)[2][Tq * G_:]                   # [n - rows, n]
    v = null.T @ np.random.default_rng(seed).standard_normal((len(null), 64))
    v = torch.from_numpy(v / np.abs(v).max()).to(BF16)
    for j in range(n):
        bt.pages[1][int(bt.table[0, j // 16]), 0, j % 16] = v[j]
    return bt, q, parents, p, to64(v)


CASES = [(120, 8, 4, 90, 3, False), (90, 17, 1, 2**30, 0, False), (150, 5, 5, 0, 0, True),
         (200, 20, 1, 0, 0, True), (130, 2, 16, 100, 9, False)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_one_rounding_to_bf16_would_be_seen(monkeypatch, case):
    """The same tolerances on the host: weights of two bf16 parts keep them, of one do not."""
    monkeypatch.setattr(M, "FEW_ROWS", 32)
    bt, q, parents, p, v = cancelling(*CASES[case], seed=1600 + case)
    ref, tol = masked_reference(q, bt, 0.25, CASES[case][3], CASES[case][4], parents)
    one = to64(torch.from_numpy(p).to(BF16))
    two = one + to64(torch.from_numpy(p - one).to(BF16))
    for w, fits in ((one, False), (two, True)):
        o = to64(torch.from_numpy(w @ v).to(BF16)).reshape(ref.shape)
        assert (np.abs(o - ref) <= tol).all() == fits


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_seventeen_to_32_rows_of_heads_of_64(rf, monkeypatch, case):  # noqa: F811
    monkeypatch.setattr(M, "FEW_ROWS", 32)
    bt, q, parents, _, _ = cancelling(*CASES[case], seed=1600 + case)
    assert 16 < q.shape[1] * q.shape[2] <= 32
    window, sinks = CASES[case][3:5]
    got, status = run(rf, bt, q, 0.25, window, sinks, parents)
    assert status == rf.RF_OK
    ref, tol = masked_reference(q, bt, 0.25, window, sinks, parents)
    err = np.abs(to64(got) - ref)
    assert (err <= tol).all(), f"{CASES[case]}: worst {(err / tol).max():.2f} of the tolerance"
