"""Prompts with a sliding window and sinks (rf_attn_fwd_window) on the GPU against the
fp64 oracle.

Tolerance: one rounding to bf16 (half a step, 2^-8 relative) of a sum of weights times
values in which every weight carries its rounding to bf16 (2^-8), the error of its score
(an fp32 sum of d products, a product and the exponential) and that of the running sums.
"""
import functools

import numpy as np
import pytest
import torch

from oracle import paged as G
from tests.helpers import Guarded, to64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    assert torch.cuda.is_available()
    assert m.rf_get_device_status() == m.RF_OK
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cu(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32)


def reference(q, k, v, new, keys, scale, window, sinks, pad_q=0):
    """(o, tolerance) in fp64, a sequence and kv head at a time."""
    q, k, v = to64(q), to64(k), to64(v)
    d, G_ = q.shape[2], q.shape[1] // k.shape[1]
    o, tol = np.zeros_like(q), np.zeros_like(q)
    u = 2.0 ** -23
    q0 = k0 = 0
    for n, nk in zip(new, keys):
        pos = np.arange(n)[:, None] + nk - n
        j = np.arange(nk)[None]
        seen = j <= pos
        if window:
            seen = seen & ((pos - j < window) | (j < sinks))
        for h in range(k.shape[1] if n and nk else 0):
            kb, vb = k[k0:k0 + nk, h], v[k0:k0 + nk, h]
            for hq in range(h * G_, (h + 1) * G_):
                x = q[q0:q0 + n, hq]
                s = np.where(seen, scale * x @ kb.T, -np.inf)
                size = np.where(seen, scale * np.abs(x) @ np.abs(kb).T, 0).max(1)
                top = s.max(1, keepdims=True)
                p = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0)), 0)
                p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
                big = np.abs(np.where(seen, s, 0)).max(1)
                e = (d + 8) * u * size + 4 * u * big + 8 * u
                per = 2 * e + 2.0 ** -8 + (seen.sum(1) / 8 + 64) * u
                o[q0:q0 + n, hq] = p @ vb
                tol[q0:q0 + n, hq] = per[:, None] * (p @ np.abs(vb))
        q0, k0 = q0 + n, k0 + nk
    return o, tol + 2.0 ** -8 * (np.abs(o) + tol) + 1e-37


def assert_close(got, ref, tol, what):
    got = to64(got)
    assert np.isfinite(got).all(), what
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside; worst "
                           f"{(np.abs(got - ref) / tol).max():.2f} of the tolerance")


def inputs(new, keys, Hq, Hkv, d, seed):
    g = _gen(seed)
    q = torch.randn(sum(new), Hq, d, generator=g).to(BF16)
    k, v = (torch.randn(sum(keys), Hkv, d, generator=g).to(BF16) for _ in range(2))
    return q, k, v


CASES = [
    # d, Hq, Hkv, window, sinks, new tokens, keys (None: the same)
    (64, 2, 2, 16, 0, [1, 5, 128, 129, 0, 200], None),
    (128, 8, 2, 16, 4, [1, 5, 31, 32, 33, 64, 65, 200], None),
    (128, 2, 2, 130, 1, [300, 1], None),
    (64, 8, 1, 1, 0, [70, 3], None), (128, 4, 1, 1, 2, [70, 3], None),
    (128, 5, 1, 40, 3, [200, 26, 25, 24], None), (64, 14, 2, 128, 128, [400], None),
    (128, 16, 1, 100, 300, [600], None), (64, 128, 1, 7, 2, [50], None),
    (128, 100, 1, 7, 2, [20], None), (64, 66, 1, 30, 0, [9, 90], None),
    (128, 4, 4, 0, 0, [500, 77], None), (64, 6, 3, 0, 9, [300, 1, 140], None),
    # earlier keys in front of the new tokens, aligned and not
    (128, 8, 2, 64, 4, [100, 1, 50, 7], [500, 1000, 129, 8]),
    (64, 2, 1, 200, 130, [64, 33, 1], [640, 1000, 131]),
    (128, 4, 2, 1000, 0, [256, 10], [900, 1010]), (64, 4, 1, 0, 0, [130, 1], [400, 257]),
    # fewer keys than tokens: the first rows read nothing; none at all
    (128, 4, 1, 16, 2, [100, 40, 30], [60, 0, 1]), (64, 2, 2, 0, 0, [300, 3], [10, 0]),
    # far sinks beside far windows
    (128, 8, 2, 300, 1, [1200], [3000]), (64, 8, 8, 128, 260, [900], [2000]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_prompts(rf, case):
    d, Hq, Hkv, window, sinks, new, keys = CASES[case]
    keys = keys or new
    q, k, v = inputs(new, keys, Hq, Hkv, d, case)
    o = Guarded(tuple(q.shape), BF16)
    rf.rf_attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), o.t, d ** -0.5, window, sinks, _cu(new).cuda(),
                          _cu(keys).cuda(), max(new))
    assert rf.rf_get_device_status() == rf.RF_OK
    o.check("output")
    assert_close(o.t, *reference(q, k, v, new, keys, d ** -0.5, window, sinks), CASES[case])


def test_reference_is_the_oracle_of_every_row():
    new, keys = [7, 2], [20, 9]
    q, k, v = inputs(new, keys, 4, 2, 16, 5)
    for window, sinks in ((0, 0), (4, 2), (1, 0)):
        np.testing.assert_allclose(reference(q, k, v, new, keys, 0.3, window, sinks)[0],
                                   G.window_prompt(q, k, v, new, keys, 0.3, window, sinks), atol=1e-12)


@pytest.mark.parametrize("d", [64, 128])
def test_long_prompts_in_many_items(rf, d):
    """More items than CTAs, ragged, with sequences that have none."""
    new = [1500, 0, 7, 900, 2300, 0, 64]
    q, k, v = inputs(new, new, 8, 4, d, 40)
    o = Guarded(tuple(q.shape), BF16)
    cu = _cu(new).cuda()
    rf.rf_attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), o.t, d ** -0.5, 333, 5, cu, cu, 2300)
    assert rf.rf_get_device_status() == rf.RF_OK
    o.check("output")
    assert_close(o.t, *reference(q, k, v, new, new, d ** -0.5, 333, 5), d)


def test_views_of_a_fused_projection_and_rows_left_alone(rf):
    """Strided tokens on every side; what lies between and behind them stays."""
    n, Hq, Hkv, d = 150, 6, 2, 64
    qkv = torch.randn(n, Hq + 2 * Hkv, d, generator=_gen(50)).to(BF16)
    dev = qkv.cuda()
    wide = torch.full((n + 20, Hq + 3, d), 7.0, dtype=BF16, device="cuda")
    cu = _cu([90, 60]).cuda()
    rf.rf_attn_fwd_window(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], wide[:n, 1:Hq + 1], 0.125, 20,
                          3, cu, cu, 90)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    assert_close(wide[:n, 1:Hq + 1], *reference(q, k, v, [90, 60], [90, 60], 0.125, 20, 3), "views")
    assert (wide[:, 0] == 7).all() and (wide[:, Hq + 1:] == 7).all() and (wide[n:] == 7).all()
    assert torch.equal(dev.cpu(), qkv)
    # tokens behind the last sequence: their rows are not written
    o = torch.full((n, Hq, d), 7.0, dtype=BF16, device="cuda")
    cu = _cu([90, 20]).cuda()
    rf.rf_attn_fwd_window(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], o, 0.125, 20, 3, cu, cu, 90)
    assert (o[110:] == 7).all()
    assert_close(o[:110], *reference(q[:110], k, v, [90, 20], [90, 20], 0.125, 20, 3), "fewer tokens")
    assert rf.rf_get_device_status() == rf.RF_OK


def test_equal_lengths_without_cumulative_ones(rf):
    new, keys = [40] * 3, [70] * 3
    q, k, v = (t.cuda() for t in inputs(new, keys, 4, 2, 128, 60))
    outs = []
    for cq, ck in ((None, None), (_cu(new).cuda(), None), (None, _cu(keys).cuda()),
                   (_cu(new).cuda(), _cu(keys).cuda())):
        o = torch.empty_like(q)
        rf.rf_attn_fwd_window(q, k, v, o, 0.1, 25, 2, cq, ck, 40 if cq is not None else None, batch=3)
        outs.append(o)
    assert all(torch.equal(o, outs[0]) for o in outs)
    assert_close(outs[0], *reference(q, k, v, new, keys, 0.1, 25, 2), "equal lengths")
    # one sequence, nothing else said
    o = torch.empty_like(q)
    rf.rf_attn_fwd_window(q, k, v, o, 0.1, 25)
    assert_close(o, *reference(q, k, v, [120], [210], 0.1, 25, 0), "one sequence")


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("d,Hq", [(64, 1), (128, 4)])
def test_values_that_are_not_finite_reach_only_the_rows_that_read_them(rf, which, d, Hq):
    new, keys, window, sinks = [200, 70], [260, 70], 50, 3
    q, k, v = inputs(new, keys, Hq, 1, d, 70)
    ref, tol = reference(q, k, v, new, keys, 0.1, window, sinks)
    for b, key, x in ((0, 0, "inf"), (0, 2, "nan"), (0, 3, "nan"), (0, 61, "inf"), (0, 130, "-inf"),
                      (0, 259, "inf"), (1, 0, "nan"), (1, 69, "inf"), (1, 33, "inf")):
        kk, vv = k.clone(), v.clone()
        row = (kk if which == "k" else vv)[260 * b + key, 0]
        row[5 if which == "v" else slice(None)] = float(x)
        o = torch.empty(q.shape, dtype=BF16, device="cuda")
        rf.rf_attn_fwd_window(q.cuda(), kk.cuda(), vv.cuda(), o, 0.1, window, sinks, _cu(new).cuda(),
                              _cu(keys).cuda(), 200)
        assert rf.rf_get_device_status() == rf.RF_OK
        got = to64(o)
        for c, n in enumerate(new):
            pos = np.arange(n) + keys[c] - n
            reads = (c == b) & (key <= pos) & ((pos - key < window) | (key < sinks))
            rows = slice(200 * c, 200 * c + n)
            g_, r_, t_ = got[rows], ref[rows], tol[rows]
            assert (np.abs(g_ - r_) <= t_)[~reads].all(), f"rows that do not read key {key} of {b}"
            if which == "v":
                assert not np.isfinite(g_[reads][..., 5]).any(), f"rows that read key {key} of {b}"
                other = np.arange(d) != 5
                assert (np.abs(g_ - r_) <= t_)[reads][..., other].all(), "the other dims of those rows"
                if x != "nan":
                    assert (g_[reads][..., 5] == float(x)).all()
            elif reads.any():
                assert not np.isfinite(g_[reads]).all(-1).any()


def test_scores_of_minus_infinity_and_of_great_size(rf):
    """Rows all of whose scores are -infinity are zeros; large scores pick their key."""
    n, d = 100, 64
    q = torch.zeros(n, 1, d, dtype=BF16)
    k = torch.zeros(n, 1, d, dtype=BF16)
    v = torch.randn(n, 1, d, generator=_gen(80)).to(BF16)
    q[..., 0] = 1
    k[:30, 0, 0] = float("-inf")
    o = torch.empty(q.shape, dtype=BF16, device="cuda")
    rf.rf_attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), o, 1.0, 10)
    got = to64(o)
    assert not got[:30].any()
    kk = k.clone()
    kk[:30] = 0
    keep = np.arange(n) >= 40                               # their windows have none of the thirty
    ref, tol = reference(q, kk, v, [n], [n], 1.0, 10, 0)
    assert (np.abs(got - ref) <= tol)[keep].all()
    k = torch.zeros(n, 1, d, dtype=BF16)
    k[::7, 0, 0] = 3000
    o.zero_()
    rf.rf_attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), o, 1.0, 10)
    assert_close(o, *reference(q, k, v, [n], [n], 1.0, 10, 0), "large scores")
    # scores that grow and fall along the keys, over several tiles
    m = 700
    q, k, v = inputs([m], [m], 2, 1, d, 81)
    k *= torch.linspace(0, 20, m)[:, None, None].to(BF16)
    for kk in (k, k.flip(0)):
        o = torch.empty(q.shape, dtype=BF16, device="cuda")
        rf.rf_attn_fwd_window(q.cuda(), kk.cuda(), v.cuda(), o, 0.125, 400, 8)
        assert_close(o, *reference(q, kk, v, [m], [m], 0.125, 400, 8), "growing scores")
    assert rf.rf_get_device_status() == rf.RF_OK


def test_inconsistent_lengths_are_reported_and_skipped(rf):
    new = [40, 50, 30]
    q, k, v = inputs(new, new, 2, 1, 64, 90)
    ref, tol = reference(q, k, v, new, new, 0.125, 16, 2)
    good = _cu(new)
    for name, at, x in (("q", 2, 5000), ("q", 1, -7), ("k", 2, 10**6), ("k", 1, -1)):
        cq, ck = good.clone(), good.clone()
        (cq if name == "q" else ck)[at] = x
        o = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
        rf.rf_attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), o, 0.125, 16, 2, cq.cuda(), ck.cuda(), 50)
        assert rf.rf_get_device_status() == rf.RF_ERR_DEVICE_INPUT
        for b in range(3):
            rows = slice(int(good[b]), int(good[b + 1]))
            if b in (at - 1, at):                           # the sequences next to the bad entry
                assert (o[rows] == 7).all()
            else:
                assert (np.abs(to64(o[rows]) - ref[rows]) <= tol[rows]).all()
    # a sequence longer than max_seqlen_q says
    o = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
    rf.rf_attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), o, 0.125, 16, 2, good.cuda(), good.cuda(), 45)
    assert rf.rf_get_device_status() == rf.RF_ERR_DEVICE_INPUT
    assert (o[40:90] == 7).all() and (np.abs(to64(o[:40]) - ref[:40]) <= tol[:40]).all()


def test_agrees_with_the_causal_calls_of_the_library(rf):
    """Without a window, and with one as long as the prompt, on the heads that
    rf_attn_fwd_varlen covers: both are within 2e-2 and 5e-3 of the exact result."""
    new = [300, 41]
    q, k, v = (t.cuda() for t in inputs(new, new, 4, 4, 64, 95))
    cu = _cu(new).cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    rf.rf_attn_fwd_varlen(q, k, v, a, cu, cu, 300, 0.125, 1)
    for window in (0, 300):
        rf.rf_attn_fwd_window(q, k, v, b, 0.125, window, 0, cu, cu, 300)
        assert (a.float() - b.float()).abs().max() <= 4e-2
        assert (a.double() - b.double()).norm() <= 1e-2 * a.double().norm()
    assert rf.rf_get_device_status() == rf.RF_OK


def test_repeatable_in_a_graph_and_on_other_streams(rf):
    new = [700, 33, 0, 400]
    q, k, v = (t.cuda() for t in inputs(new, new, 8, 2, 128, 100))
    cu = _cu(new).cuda()
    call = functools.partial(rf.rf_attn_fwd_window, q, k, v)
    first = torch.empty_like(q)
    call(first, 0.1, 150, 4, cu, cu, 700)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in streams]
    for _ in range(5):
        for s, o in zip(streams, outs):
            call(o, 0.1, 150, 4, cu, cu, 700, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    o = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o, 0.1, 150, 4, cu, cu, 700)
    for other in ([700, 33, 0, 400], [1, 500, 600, 32]):    # the graph follows the lengths
        cu.copy_(_cu(other))
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert_close(o, *reference(q, k, v, other, other, 0.1, 150, 4), other)
    assert rf.rf_get_device_status() == rf.RF_OK


def test_offsets_beyond_32_bits(rf):
    """Tokens 2^23 elements apart: 600 of them span 5 * 10^9 elements."""
    n, d, ld = 600, 64, 1 << 23
    base = torch.zeros(n * ld, dtype=BF16, device="cuda")
    k, v = (base[i * d:].as_strided((n, 1, d), (ld, d, 1)) for i in range(2))
    q, kk, vv = inputs([n], [n], 2, 1, d, 110)
    k.copy_(kk)
    v.copy_(vv)
    far = base[2 * d:].as_strided((n, 2, d), (ld, d, 1))
    far.copy_(q)
    rf.rf_attn_fwd_window(far, k, v, far, 0.125, 100, 2)    # in place, too
    assert_close(far, *reference(q, kk, vv, [n], [n], 0.125, 100, 2), "far tokens")
    assert rf.rf_get_device_status() == rf.RF_OK


def test_prompt_then_steps_over_the_cache(rf):
    """A windowed prompt, its append, then windowed steps over the cache: the last rows
    of the prompt equal the steps'."""
    Hq, Hkv, d, n, window, sinks = 8, 2, 128, 300, 64, 4
    q, k, v = (t.cuda() for t in inputs([n], [n], Hq, Hkv, d, 120))
    o = torch.empty_like(q)
    rf.rf_attn_fwd_window(q, k, v, o, d ** -0.5, window, sinks)
    pages = [torch.zeros(20, Hkv, 16, d, dtype=BF16, device="cuda") for _ in range(2)]
    table = torch.randperm(20, generator=_gen(121)).to(torch.int32)[None].cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cache = rf.rf_paged_kv(pages[0], pages[1], table, lens)
    rf.rf_kv_append_paged(cache, k, v)
    mask = rf.rf_attn_mask(window, sinks)
    for Tq in (1, 3, 40):
        ws = torch.empty(rf.rf_attn_decode_paged_ex_workspace_size(1, Hq, Hkv, Tq, d), dtype=torch.uint8,
                         device="cuda")
        od = torch.empty(1, Tq, Hq, d, dtype=BF16, device="cuda")
        rf.rf_attn_decode_paged_ex(cache, q[None, -Tq:].contiguous(), od, d ** -0.5, mask, ws)
        ref, tol = reference(q[-Tq:], k, v, [Tq], [n], d ** -0.5, window, sinks)
        assert_close(od[0], ref, tol, f"{Tq} tokens over the cache")
        assert_close(o[-Tq:], ref, tol, f"{Tq} tokens of the prompt")
    assert rf.rf_get_device_status() == rf.RF_OK


def test_binding_checks(rf):
    q = torch.zeros(6, 4, 64, dtype=BF16, device="cuda")
    k = torch.zeros(6, 2, 64, dtype=BF16, device="cuda")
    cu = _cu([6]).cuda()
    call = rf.rf_attn_fwd_window
    for f in (lambda: call(q.float(), k, k, q, 0.1, 4), lambda: call(q, k.cpu(), k, q, 0.1, 4),
              lambda: call(q, k, k[:5], q, 0.1, 4), lambda: call(q, k, k[:, :1], q, 0.1, 4),
              lambda: call(q, k, k, q[:5], 0.1, 4), lambda: call(q, k, k, q, 0.1, 4, 0, cu, cu),
              lambda: call(q, k, k, q, 0.1, 4, 0, cu.long(), cu, 6), lambda: call(q[0], k, k, q, 0.1, 4),
              lambda: call(q, k, k, q, 0.1, 4, 0, cu, _cu([3, 3]).cuda(), 6),
              lambda: call(q.transpose(1, 2), k, k, q, 0.1, 4), lambda: call(q, k, k, q, 0.1, 4, 0, cu[:1])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: call(q, k, k, q, 0.1, -1), lambda: call(q, k, k, q, 0.1, 4, -1),
              lambda: call(q, k, k, q, 0.0, 4), lambda: call(q, k, k, q, 0.1, 4, batch=5),
              lambda: call(q, k, k, q, 0.1, 4, batch=0), lambda: call(q[:, :3], k, k, q[:, :3], 0.1, 4),
              lambda: call(q, k, k, q, 0.1, 4, 0, cu, cu, 7)):
        with pytest.raises(rf.RFError):
            f()
    assert rf.rf_get_device_status() == rf.RF_OK
