"""Masked attention over a paged cache (windows with sinks, trees of drafted tokens)
on the GPU against the fp64 oracle.

Tolerances as in tests/test_gpu_paged.py (its head derives them), over the keys that
a row reads.  Where the weights are rounded to one 16-bit part, as the header says for
many query rows, a weight is off by half a step of that type: 2^-8 in bf16.
"""
import functools

import numpy as np
import pytest
import torch

from oracle import paged as G
from tests.helpers import Guarded, to64
from tests.test_gpu_paged import BF16, Batch, _gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    assert torch.cuda.is_available()
    assert m.rf_get_device_status() == m.RF_OK
    return m


# Above this many query rows a kv head, a bf16 cache's weights are rounded to bf16.
FEW_ROWS = 16


def half_of_a_weight(kind, rows):
    """Half a step of a rounded weight: f16 (E4M3), two bf16 parts, or one."""
    return 2.0 ** -11 if kind == "e4m3" else (2.0 ** -16 if rows <= FEW_ROWS else 2.0 ** -8)


def masked_reference(q, bt, scale, window=0, sinks=0, parents=None, lens=None, floor=2.0 ** -25,
                     below=2.0 ** -14, more=0.0):
    """(o, tolerance) in fp64; the sum of the error bounds that the file's head names.
    E4M3: weights below `below` of the row's largest are off by `floor` of it; `more` is
    a further relative error of a weight."""
    q = to64(q)
    B, Tq, Hq, d = q.shape
    K, V = (G.values(*bt.host(i)) for i in (0, 1))
    e4m3 = bt.kind == "e4m3"
    G_ = Hq // bt.Hkv
    o, tol = np.zeros_like(q), np.zeros_like(q)
    u = 2.0 ** -23
    for b, n in enumerate(bt.lens if lens is None else lens):
        if n <= 0:
            continue
        seen = [G.seen_keys(n, Tq, t, window, sinks, None if parents is None else parents[b])
                for t in range(Tq)]
        for h in range(bt.Hkv):
            for t in range(Tq):
                j = np.array(seen[t], int)
                if not len(j):
                    continue
                page = bt.table[b].numpy()[j // bt.ps]
                kb, vb = (x[page, h, j % bt.ps] for x in (K, V))
                vs = bt.scale[1][page, h] if e4m3 else np.ones(len(j))
                rows = slice(h * G_, (h + 1) * G_)
                qr = q[b, t, rows]
                s = scale * qr @ kb.T
                size = scale * np.abs(qr) @ np.abs(kb).T
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                va = np.abs(vb)
                e = (d + 8) * u * size.max(1) + 4 * u * np.abs(s).max(1) + 8 * u
                per = 2 * e + half_of_a_weight(bt.kind, Tq * G_) + (len(j) / 8 + 64) * u + more
                o[b, t, rows] = p @ vb
                tol[b, t, rows] = per[:, None] * (p @ va)
                if e4m3:
                    w = p * vs
                    top = w.max(1, keepdims=True)
                    small = w < below * top
                    tol[b, t, rows] += floor * top * (small @ (va / vs[:, None]))
    return o, tol + 2.0 ** -8 * (np.abs(o) + tol) + 1e-37


def run(rf, bt, q, scale, window=0, sinks=0, parents=None, cache=None, ws=None):
    cache = cache or bt.device(rf)
    B, Tq, Hq, d = q.shape
    o = Guarded((B, Tq, Hq, d), BF16)
    ws = ws or Guarded((rf.rf_attn_decode_paged_ex_workspace_size(B, Hq, bt.Hkv, Tq, d),), torch.uint8,
                       fill=0xFF)
    mask = rf.rf_attn_mask(window, sinks, None if parents is None else
                           torch.tensor(parents, dtype=torch.int32).cuda())
    rf.rf_attn_decode_paged_ex(cache, q.cuda(), o.t, scale, mask, ws.t)
    status = rf.rf_get_device_status()
    o.check("output")
    ws.check("workspace")
    return o.t, status


def check(rf, bt, q, scale, window=0, sinks=0, parents=None, what=""):
    got, status = run(rf, bt, q, scale, window, sinks, parents)
    assert status == rf.RF_OK, what
    ref, tol = masked_reference(q, bt, scale, window, sinks, parents)
    got = to64(got)
    assert np.isfinite(got).all(), what
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside; worst "
                           f"{(np.abs(got - ref) / tol).max():.2f} of the tolerance")
    return got


def hide_unread_pages(bt, Tq, window, sinks):
    """Entries of pages in which no row reads a key become anything."""
    for b, n in enumerate(bt.lens):
        first = max(n - Tq, 0) - window + 1
        for i in range(-(-n // bt.ps)):
            if (i + 1) * bt.ps <= first and i * bt.ps >= sinks:
                bt.table[b, i] = [-1, 10**6, -2**31, 2**31 - 1, 0][i % 5]


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 40, 64, 65, 127, 400]
WINDOWS = [
    # kind, page size, d, Hkv, Hq, Tq, window, sinks, lens
    ("e4m3", 64, 128, 2, 8, 1, 33, 4, LENS), ("e4m3", 16, 128, 1, 5, 1, 1, 0, LENS),
    ("e4m3", 16, 64, 1, 16, 1, 100, 1, LENS), ("e4m3", 128, 64, 2, 2, 1, 64, 200, LENS),
    ("bf16", 32, 64, 2, 6, 1, 16, 17, LENS), ("bf16", 16, 128, 1, 7, 1, 31, 0, LENS),
    ("bf16", 64, 64, 1, 1, 1, 128, 32, LENS), ("e4m3", 32, 128, 1, 8, 4, 20, 3, LENS),
    ("bf16", 16, 64, 2, 8, 3, 2, 1, LENS), ("e4m3", 16, 64, 1, 2, 7, 48, 0, LENS),
    ("bf16", 64, 128, 1, 4, 40, 10, 5, LENS), ("e4m3", 64, 128, 1, 4, 40, 60, 40, LENS),
    ("e4m3", 32, 64, 1, 9, 9, 1, 33, LENS), ("bf16", 128, 128, 2, 10, 33, 1000, 0, LENS),
    # long: windows cut between warps and CTAs
    ("e4m3", 64, 128, 2, 8, 1, 9000, 4, [30000, 100, 12000]),
    ("bf16", 32, 128, 1, 8, 2, 20000, 300, [25000]),
    ("e4m3", 16, 128, 1, 12, 3, 5000, 0, [15000, 9, 6000]),
    ("bf16", 16, 64, 4, 8, 1, 200, 8, [(37 * i) % 900 for i in range(90)]),
]


@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_window(rf, case):
    kind, ps, d, Hkv, Hq, Tq, window, sinks, lens = WINDOWS[case]
    bt = Batch(kind, lens, Hkv, d, ps, seed=case).garbage()
    hide_unread_pages(bt, Tq, window, sinks)
    q = torch.randn(len(lens), Tq, Hq, d, generator=_gen(100 + case)).to(BF16)
    check(rf, bt, q, d ** -0.5, window, sinks, what=f"window {WINDOWS[case][:8]}")


def tree_of(g, Tq, roots=1):
    back = (1 + torch.rand(Tq, generator=g).pow(2) * 6).long().tolist()
    return [-1 if t < roots else max(0, t - back[t]) for t in range(Tq)]


TREES = [
    # kind, page size, d, Hkv, Hq, Tq, roots, window, sinks, lens
    ("e4m3", 64, 128, 2, 8, 8, 1, 0, 0, [8, 9, 40, 64, 200]),
    ("e4m3", 16, 64, 1, 3, 5, 2, 0, 0, [5, 0, 16, 17, 33, 100]),
    ("bf16", 32, 64, 1, 4, 4, 4, 0, 0, [4, 35, 36, 37, 64]),
    ("bf16", 16, 128, 2, 4, 7, 1, 0, 0, [7, 30, 31, 32, 300]),
    ("e4m3", 32, 128, 1, 8, 17, 1, 0, 0, [17, 48, 49, 200]),
    ("bf16", 64, 128, 1, 8, 64, 1, 0, 0, [64, 128, 500, 0]),
    ("e4m3", 64, 64, 2, 8, 33, 3, 0, 0, [33, 64, 65, 700]),
    ("e4m3", 128, 128, 1, 5, 40, 1, 0, 0, [1000]),
    ("e4m3", 16, 128, 1, 4, 12, 1, 9, 2, [12, 30, 64, 100]),
    ("bf16", 32, 64, 2, 4, 25, 2, 6, 40, [25, 64, 130]),
    ("bf16", 64, 128, 1, 16, 20, 1, 100, 4, [20, 500]),
    ("e4m3", 16, 64, 1, 1, 100, 1, 3, 0, [100, 400]),
    ("e4m3", 64, 128, 1, 4, 16, 1, 0, 0, [20000, 300, 7000]),
    ("bf16", 64, 128, 2, 8, 64, 1, 0, 0, [9000, 64]),
    ("bf16", 16, 64, 2, 14, 19, 1, 4000, 4, [9000, 20]),
]


@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(rf, case):
    kind, ps, d, Hkv, Hq, Tq, roots, window, sinks, lens = TREES[case]
    g = _gen(200 + case)
    bt = Batch(kind, lens, Hkv, d, ps, seed=300 + case).garbage()
    if window:
        hide_unread_pages(bt, Tq, window, sinks)
    q = torch.randn(len(lens), Tq, Hq, d, generator=g).to(BF16)
    parents = [tree_of(g, Tq, roots) for _ in lens]
    check(rf, bt, q, d ** -0.5, window, sinks, parents, what=f"tree {TREES[case][:9]}")


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_reference_is_the_oracle_of_every_row(rf, kind):
    bt = Batch(kind, [9, 40, 0], 2, 64, 16, seed=240)
    q = torch.randn(3, 4, 4, 64, generator=_gen(241)).to(BF16)
    k, ks = bt.host(0)
    v, vs = bt.host(1)
    tree = [[-1, 0, 0, 2], [-1, -1, 1, 2], [-1, 0, 1, 2]]
    for window, sinks, parents in ((0, 0, tree), (5, 2, None), (2, 6, tree)):
        ref = G.decode_masked(q, k, v, ks, vs, bt.table.numpy(), bt.lens, 0.125, window, sinks, parents)
        np.testing.assert_allclose(masked_reference(q, bt, 0.125, window, sinks, parents)[0], ref, atol=1e-12)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_masks_that_hide_nothing_give_what_no_mask_gives(rf, kind):
    """A null mask is the unmasked call, bit for bit; a window beyond the longest
    sequence and a tree that is a chain agree with it within both tolerances."""
    bt = Batch(kind, [50, 3, 0, 300], 2, 128, 32, seed=5).garbage()
    q = torch.randn(4, 3, 8, 128, generator=_gen(6)).to(BF16)
    cache = bt.device(rf)
    ws = torch.empty(rf.rf_attn_decode_paged_ex_workspace_size(4, 8, 2, 3, 128), dtype=torch.uint8,
                     device="cuda")
    qd = q.cuda()
    a, b = torch.empty_like(qd), torch.empty_like(qd)
    rf.rf_attn_decode_paged(cache, qd, a, 0.0884, ws)
    for mask in (None, rf.rf_attn_mask(), rf.rf_attn_mask(0, 7)):
        rf.rf_attn_decode_paged_ex(cache, qd, b.fill_(7), 0.0884, mask, ws)
        assert torch.equal(a, b)
    for window, sinks, parents in ((2**30, 2**30, None), (300, 0, None), (0, 0, [[-1, 0, 1]] * 4)):
        if parents is not None:
            bt.lens = [50, 3, 0, 300]
        check(rf, bt, q, 0.0884, window, sinks, parents, what="hides nothing")


ODD_VALUES = [(kind, Tq, Hq, tree) for kind in ("e4m3", "bf16")
              for Tq, Hq, tree in ((1, 4, False), (3, 2, False), (6, 4, True), (20, 8, True), (20, 8, False))]


@pytest.mark.parametrize("kind,Tq,Hq,tree", ODD_VALUES)
def test_values_that_are_not_finite_reach_only_the_rows_that_read_them(rf, kind, Tq, Hq, tree):
    """An infinity or NaN in a key or value, anywhere in the sequence: before the
    window, at its border, among the nodes."""
    n, window, sinks = 90, 30, 5
    bt = Batch(kind, [n], 1, 64, 16, seed=260)
    clean = bt.pages.copy() if kind == "e4m3" else bt.pages.clone()
    q = torch.randn(1, Tq, Hq, 64, generator=_gen(261)).to(BF16)
    parents = [tree_of(_gen(Tq), Tq)] if tree else None
    ref, tol = masked_reference(q, bt, 0.125, window, sinks, parents)
    seen = [G.seen_keys(n, Tq, t, window, sinks, parents[0] if tree else None) for t in range(Tq)]
    for key in (0, sinks, 20, n - Tq - window, n - Tq - window + 2, n - window, n - Tq, n - 2, n - 1):
        if key < 0:
            continue
        for which in (0, 1):
            bt.pages = clean.copy() if kind == "e4m3" else clean.clone()
            bt.pages[which][int(bt.table[0, key // 16]), 0, key % 16] = \
                0x7F if kind == "e4m3" else float("inf")
            got, status = run(rf, bt, q, 0.125, window, sinks, parents)
            assert status == rf.RF_OK
            got = to64(got)
            for t in range(Tq):
                if key in seen[t]:
                    assert not np.isfinite(got[0, t]).all(-1).any(), f"row {t} reads key {key}"
                else:
                    assert (np.abs(got - ref) <= tol)[0, t].all(), f"row {t} does not read key {key}"


@pytest.mark.parametrize("kind,Tq,Hq", [("e4m3", 6, 4), ("bf16", 6, 2), ("bf16", 24, 4)])
def test_bad_trees_are_reported_and_their_rows_are_zeros(rf, kind, Tq, Hq):
    lens = [50, Tq - 1, 70, 0, 200]
    bt = Batch(kind, lens, 1, 64, 16, seed=270)
    q = torch.randn(5, Tq, Hq, 64, generator=_gen(271)).to(BF16)
    good = [tree_of(_gen(272), Tq) for _ in lens]
    got, status = run(rf, bt, q, 0.125, parents=good)
    assert status == rf.RF_ERR_DEVICE_INPUT            # the sequence of Tq - 1 tokens
    ref, tol = masked_reference(q, bt, 0.125, parents=good)
    assert (np.abs(to64(got) - ref) <= tol).all() and not got[1].any() and not got[3].any()
    for bad in (-2, Tq, 3, 2**31 - 1, -2**31):
        parents = [list(p) for p in good]
        parents[2][3] = bad
        bt.lens = [50, 0, 70, 0, 200]
        got, status = run(rf, bt, q, 0.125, parents=parents)
        assert status == rf.RF_ERR_DEVICE_INPUT
        ref, tol = masked_reference(q, bt, 0.125, parents=parents)
        assert (np.abs(to64(got) - ref) <= tol).all() and not got[2, 3].any()
        bt.lens = lens


def test_a_page_outside_the_cache_within_the_window_is_reported(rf):
    bt = Batch("bf16", [100, 100], 1, 64, 16, seed=280)
    q = torch.randn(2, 1, 4, 64, generator=_gen(281)).to(BF16)
    ok = bt.table.clone()
    bt.table[0, 2] = bt.num_pages                      # keys 32 .. 47: not read
    assert run(rf, bt, q, 0.125, 40, 4)[1] == rf.RF_OK
    bt.table[0, 0] = -1                                # the sinks
    got, status = run(rf, bt, q, 0.125, 40, 4)
    assert status == rf.RF_ERR_DEVICE_INPUT
    bt.table = ok
    ref, tol = masked_reference(q, bt, 0.125, 40, 0)   # sequence 0 without its sinks
    full, ftol = masked_reference(q, bt, 0.125, 40, 4)
    assert (np.abs(to64(got) - ref) <= tol)[0].all() and (np.abs(to64(got) - full) <= ftol)[1].all()


def test_in_place_and_repeatable(rf):
    for kind, Tq in (("e4m3", 1), ("bf16", 48)):
        bt = Batch(kind, [5000, 100, 2500], 2, 128, 64, seed=290)
        cache = bt.device(rf)
        q = torch.randn(3, Tq, 8, 128, generator=_gen(291)).to(BF16).cuda()
        ws = torch.empty(rf.rf_attn_decode_paged_ex_workspace_size(3, 8, 2, Tq, 128), dtype=torch.uint8,
                         device="cuda")
        mask = rf.rf_attn_mask(2000, 4)
        first = torch.empty_like(q)
        rf.rf_attn_decode_paged_ex(cache, q, first, 0.0884, mask, ws)
        for _ in range(8):
            ws.random_(0, 256)
            o = q.clone()
            rf.rf_attn_decode_paged_ex(cache, o, o, 0.0884, mask, ws)
            assert torch.equal(o, first)
        with pytest.raises(rf.RFError) as e:
            rf.rf_attn_decode_paged_ex(cache, q, first, 0.0884, mask, ws[:ws.numel() - 16])
        assert e.value.status == rf.RF_ERR_WORKSPACE
    assert rf.rf_get_device_status() == rf.RF_OK


@pytest.mark.parametrize("Tq", [6, 12])
def test_draft_verify_accept_in_a_graph(rf, Tq):
    """A drafting loop: norm and rotation of the nodes at their depths, append, attention
    over the tree; the accepted line is appended again behind the context and the next tree
    follows.  Captured once, replayed with trees, lengths and positions that change; each
    step equals the oracle's for the cache it left."""
    B, Hq, Hkv, d, ps, window = 2, 4, 1, 64, 16, 50
    bt = Batch("bf16", [300, 300], Hkv, d, ps, seed=500)
    cache = bt.device(rf, [40, 61])
    a = torch.arange(400, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)[None, :]
    nr = rf.rf_norm_rope(a.cos().float().cuda(), a.sin().float().cuda())
    qkv = torch.zeros(B * Tq, Hq + 2 * Hkv, d, dtype=BF16, device="cuda")
    pos = torch.zeros(B * Tq, dtype=torch.int32, device="cuda")
    parents = torch.full((B, Tq), -1, dtype=torch.int32, device="cuda")
    mask = rf.rf_attn_mask(window, 4, parents)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    qr = torch.empty(B, Tq, Hq, d, dtype=BF16, device="cuda")
    kr = torch.empty(B * Tq, Hkv, d, dtype=BF16, device="cuda")
    o = torch.empty_like(qr)
    ws = torch.empty(rf.rf_attn_decode_paged_ex_workspace_size(B, Hq, Hkv, Tq, d), dtype=torch.uint8,
                     device="cuda")

    def step():
        rf.rf_qk_norm_rope(q, k, qr.view(B * Tq, Hq, d), kr, nr, pos)
        rf.rf_kv_append_paged(cache, kr, qkv[:, Hq + Hkv:])
        rf.rf_attn_decode_paged_ex(cache, qr, o, 0.125, mask, ws)

    bt.dlens.add_(Tq)
    step()                                             # the first call, before the capture
    bt.dlens.sub_(Tq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = _gen(501)
    for it in range(6):
        trees = [tree_of(g, Tq) for _ in range(B)]
        lens = bt.dlens.tolist()
        depth = [[len(G.line_of(tr, t)) - 1 for t in range(Tq)] for tr in trees]
        parents.copy_(torch.tensor(trees, dtype=torch.int32))
        pos.copy_(torch.tensor([n + x for n, row in zip(lens, depth) for x in row], dtype=torch.int32))
        qkv.copy_(torch.randn(B * Tq, Hq + 2 * Hkv, d, generator=g).to(BF16))
        bt.dlens.add_(Tq)
        graph.replay()
        torch.cuda.synchronize()
        bt.lens = bt.dlens.tolist()
        bt.pages = torch.stack([bt.k.t.cpu(), bt.v.t.cpu()])
        ref, tol = masked_reference(qr.cpu(), bt, 0.125, window, 4, trees)
        assert (np.abs(to64(o) - ref) <= tol).all(), f"step {it}"
        # accept a line: its rows again, from the first node's slot on
        take = [list(reversed(G.line_of(tr, int(torch.randint(Tq, (1,), generator=g))))) for tr in trees]
        rows = torch.tensor([b * Tq + u for b, t in enumerate(take) for u in t]).cuda()
        cu = torch.tensor([0, len(take[0]), len(take[0]) + len(take[1])], dtype=torch.int32).cuda()
        bt.dlens.copy_(torch.tensor([n + len(t) for n, t in zip(lens, take)], dtype=torch.int32))
        rf.rf_kv_append_paged(cache, kr[rows], qkv[rows, Hq + Hkv:], None, cu)
    assert rf.rf_get_device_status() == rf.RF_OK


def test_two_streams_and_a_padded_batch(rf):
    sets = []
    for i in range(2):
        bt = Batch("e4m3", [6000, 0, 300], 2, 128, 32, seed=710 + i)
        q = torch.randn(3, 4, 8, 128, generator=_gen(712 + i)).to(BF16).cuda()
        ws = torch.empty(rf.rf_attn_decode_paged_ex_workspace_size(3, 8, 2, 4, 128), dtype=torch.uint8,
                         device="cuda")
        mask = rf.rf_attn_mask(1000, 4) if i else rf.rf_attn_mask(
            0, 0, torch.tensor([[-1, 0, 0, 1]] * 3, dtype=torch.int32).cuda())
        sets.append((bt.device(rf), q, torch.empty_like(q), ws, mask, torch.cuda.Stream(), bt))
    alone = []
    for cache, q, o, ws, mask, _, _ in sets:
        rf.rf_attn_decode_paged_ex(cache, q, o, 0.0884, mask, ws)
        torch.cuda.synchronize()
        assert not o[1].any()
        alone.append(o.clone())
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for cache, q, o, ws, mask, s, _ in sets:
            rf.rf_attn_decode_paged_ex(cache, q, o, 0.0884, mask, ws, stream=s)
    torch.cuda.synchronize()
    for (_, _, o, _, _, _, _), x in zip(sets, alone):
        assert torch.equal(o, x)


def test_binding_checks(rf):
    bt = Batch("e4m3", [20, 20], 2, 64, 16, seed=720)
    cache = bt.device(rf)
    q = torch.zeros(2, 3, 4, 64, dtype=BF16, device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    par = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    call = functools.partial(rf.rf_attn_decode_paged_ex, cache, q, q.clone(), 0.1)
    for f in (lambda: rf.rf_attn_mask(-1), lambda: rf.rf_attn_mask(5, -1), lambda: rf.rf_attn_mask(2**30 + 1),
              lambda: rf.rf_attn_mask(0, 0, par.long()), lambda: rf.rf_attn_mask(0, 0, par.cpu()),
              lambda: rf.rf_attn_mask(0, 0, par[0]), lambda: rf.rf_attn_mask(0, 0, par.t()),
              lambda: call(rf.rf_attn_mask(0, 0, par[:1]), ws),
              lambda: call(rf.rf_attn_mask(0, 0, par[:, :2].contiguous()), ws),
              lambda: call(rf.rf_attn_mask(3), ws.cpu())):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(rf.RFError):
        call(rf.rf_attn_mask(3), None)
    assert rf.rf_get_device_status() == rf.RF_OK
