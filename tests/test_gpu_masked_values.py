"""Masked attention of many query rows over a paged cache at the values where it can go
wrong: weights that span many binades, scales of codes far from one and far from each
other, scores of great size; bad trees, bad pages, reuse and several streams there.

Tolerances as in tests/test_gpu_masked.py.  Of E4M3's weights (times their value scale),
rounded to f16, the largest of a row is at least 2^7 when it is rounded, so one below
2^-21 of it lies below f16's normal numbers and is off by at most 2^-25 / 2^7 = 2^-32 of
it.  With scales that are no powers of two a weight's exponent is a sum with log2 of its
scale, of at most 2^7 in size here: three roundings of 2^-18 each, and the logarithm's own
2^-21, times ln 2.
"""
import numpy as np
import pytest
import torch

from tests import test_gpu_masked as M
from tests.helpers import to64
from tests.test_gpu_masked import masked_reference, rf, run, tree_of  # noqa: F401
from tests.test_gpu_paged import BF16, Batch, _gen
from tests.test_gpu_paged_values import _sink

pytestmark = pytest.mark.gpu

MANY = dict(floor=2.0 ** -32, below=2.0 ** -21)
EXPONENTS = 2.0 ** -16


def compare(rf, bt, q, scale, what, window=0, sinks=0, parents=None, more=0.0):  # noqa: F811
    assert q.shape[1] * q.shape[2] // bt.Hkv > (48 if bt.d == 128 else 80)     # many rows for either cache
    got, status = run(rf, bt, q, scale, window, sinks, parents)
    assert status == rf.RF_OK, what
    ref, tol = masked_reference(q, bt, scale, window, sinks, parents, more=more, **MANY)
    err = np.abs(to64(got) - ref)
    assert (err <= tol).all(), f"{what}: worst {np.nanmax(err / tol):.2f} of the tolerance"


def chain(Tq):
    return [t - 1 for t in range(Tq)]


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("gap", [4, 10, 14, 18])
@pytest.mark.parametrize("first", [0.0, 2.0 ** -7, 1.0])
@pytest.mark.parametrize("n,d,G_,Tq", [(2048, 128, 4, 16), (700, 64, 3, 28), (1000, 128, 12, 5)])
def test_a_dominant_key_does_not_drown_the_others(rf, kind, gap, first, n, d, G_, Tq):  # noqa: F811
    """The others' weights are e^-gap of the first key's, whose value is zero or small."""
    bt, q = _sink(kind, n, d, gap, first, 900 + gap, G_, Tq)
    compare(rf, bt, q, 1.0, f"gap {gap}", parents=[chain(Tq)])


@pytest.mark.parametrize("v_exp", [-114, -105, 112])
@pytest.mark.parametrize("lens", [[70, 24], [9000, 30]])
@pytest.mark.parametrize("d", [64, 128])
def test_value_scales_next_to_fp32s_ends(rf, v_exp, lens, d):  # noqa: F811
    bt = Batch("e4m3", lens, 1, d, 32, seed=930, loud=0.0)
    bt.scale[1] *= np.float32(2.0 ** v_exp)
    q = torch.randn(2, 24, 4, d, generator=_gen(931)).to(BF16)
    compare(rf, bt, q, d ** -0.5, f"value scales of 2^{v_exp}", parents=[chain(24)] * 2)


@pytest.mark.parametrize("d,ps,Tq,G_", [(128, 64, 13, 4), (128, 16, 33, 5), (64, 32, 96, 1), (64, 128, 20, 8)])
@pytest.mark.parametrize("spread", [0, 20, 60])
@pytest.mark.parametrize("odd", [False, True])
def test_scales_that_differ_from_page_to_page(rf, d, ps, Tq, G_, spread, odd):  # noqa: F811
    lens = [300, 0, Tq, 1700]
    bt = Batch("e4m3", lens, 2, d, ps, seed=940 + spread).garbage()
    g = np.random.default_rng(941)
    shape = bt.scale[1].shape
    bt.scale[1] *= np.exp2(g.integers(-spread, spread + 1, shape)).astype(np.float32)
    if odd:
        bt.scale[0] *= g.uniform(0.7, 1.4, shape).astype(np.float32)
        bt.scale[1] *= g.uniform(0.7, 1.4, shape).astype(np.float32)
    q = torch.randn(4, Tq, 2 * G_, d, generator=_gen(942)).to(BF16)
    trees = [tree_of(_gen(943 + b), Tq) for b in range(4)]
    for window, sinks, parents in ((0, 0, trees), (150, 9, None)):
        compare(rf, bt, q, d ** -0.5, f"spread {spread}", window, sinks, parents, more=EXPONENTS)


def test_pages_of_zeros(rf):  # noqa: F811
    """Codes of zero alone: the smallest normal scale is what an append gives them."""
    bt = Batch("e4m3", [200, 100], 1, 128, 16, seed=950)
    for which in (0, 1):
        for i in (0, 3, 12):
            page = int(bt.table[0, i])
            bt.pages[which][page] = 0
            bt.scale[which][page] = np.float32(2.0 ** -126)
    q = torch.randn(2, 13, 4, 128, generator=_gen(951)).to(BF16)
    compare(rf, bt, q, 0.0884, "pages of zeros", parents=[chain(13)] * 2)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("Tq,G_", [(24, 4), (30, 3)])
@pytest.mark.parametrize("exp", [4, 10, 16])
def test_scores_up_to_a_million(rf, kind, Tq, G_, exp):  # noqa: F811
    bt = Batch(kind, [500, 33], 1, 64, 16, seed=960)
    q = (torch.randn(2, Tq, G_, 64, generator=_gen(961)) * 2.0 ** exp).to(BF16)
    got, status = run(rf, bt, q, 1.0, parents=[tree_of(_gen(962), Tq)] * 2)
    assert status == rf.RF_OK
    ref, tol = masked_reference(q, bt, 1.0, parents=[tree_of(_gen(962), Tq)] * 2)
    assert (np.abs(to64(got) - ref) <= tol).all()


@pytest.mark.parametrize("exp", [-130, -60, 60, 120])
def test_queries_of_any_size(rf, exp):  # noqa: F811
    """E4M3: they are scaled to f16's range row by row."""
    bt = Batch("e4m3", [150, 33], 1, 64, 16, seed=965, loud=0.0)
    q = torch.randn(2, 30, 3, 64, generator=_gen(966)).to(BF16)
    q[:, ::3] = (q[:, ::3].float() * 2.0 ** exp).to(BF16)
    scale = 2.0 ** -max(exp, 0)                        # the products stay within fp32
    compare(rf, bt, q, scale, f"queries of 2^{exp}", parents=[chain(30)] * 2)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("window", [0, 90])
def test_trees_of_many_nodes(rf, kind, window):  # noqa: F811
    """Lines of hundreds of parents, over several key tiles."""
    bt = Batch(kind, [900, 650], 1, 64, 32, seed=968).garbage()
    q = torch.randn(2, 650, 2, 64, generator=_gen(969)).to(BF16)
    compare(rf, bt, q, 0.125, "many nodes", window, 3, [chain(650), tree_of(_gen(967), 650)])


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("Tq,Hq", [(24, 4), (45, 2)])
def test_bad_trees(rf, kind, Tq, Hq):  # noqa: F811
    M.test_bad_trees_are_reported_and_their_rows_are_zeros(rf, kind, Tq, Hq)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_bad_pages_and_lengths(rf, kind):  # noqa: F811
    """Pages outside the cache count as empty, lengths beyond the table as none."""
    Tq, lens = 20, [100, 100, 60]
    bt = Batch(kind, lens, 1, 64, 16, seed=970)
    q = torch.randn(3, Tq, 5, 64, generator=_gen(971)).to(BF16)
    full, ftol = masked_reference(q, bt, 0.125, 30, 4)
    ok = bt.table.clone()
    bt.table[0, 2] = bt.num_pages                      # keys 32 .. 47: not read
    assert run(rf, bt, q, 0.125, 30, 4)[1] == rf.RF_OK
    bt.table[0, 0] = -1                                # the sinks
    got, status = run(rf, bt, q, 0.125, 30, 4)
    assert status == rf.RF_ERR_DEVICE_INPUT
    ref, tol = masked_reference(q, bt, 0.125, 30, 0)
    assert (np.abs(to64(got) - ref) <= tol)[0].all() and (np.abs(to64(got) - full) <= ftol)[1:].all()
    bt.table = ok
    for bad in (-1, 10**6, -2**31, 2**31 - 1):
        cache = bt.device(rf, [100, bad, 60])
        got, status = run(rf, bt, q, 0.125, 30, 4, cache=cache)
        assert status == rf.RF_ERR_DEVICE_INPUT
        assert (np.abs(to64(got) - full) <= ftol)[[0, 2]].all() and not got[1].any()


def test_repeatable_in_place_on_two_streams(rf):  # noqa: F811
    sets = []
    for i, kind in enumerate(("e4m3", "bf16")):
        bt = Batch(kind, [5000, 0, 100, 2500], 2, 128, 64, seed=980 + i)
        q = torch.randn(4, 16, 8, 128, generator=_gen(981 + i)).to(BF16).cuda()
        ws = torch.empty(rf.rf_attn_decode_paged_ex_workspace_size(4, 8, 2, 16, 128), dtype=torch.uint8,
                         device="cuda")
        par = torch.tensor([tree_of(_gen(982), 16)] * 4, dtype=torch.int32).cuda()
        sets.append((bt.device(rf), q, ws, rf.rf_attn_mask(2000, 4, par), torch.cuda.Stream(), bt))
    first = []
    for cache, q, ws, mask, _, _ in sets:
        o = torch.empty_like(q)
        rf.rf_attn_decode_paged_ex(cache, q, o, 0.0884, mask, ws)
        first.append(o)
    torch.cuda.synchronize()
    for _ in range(4):
        outs = [q.clone() for _, q, _, _, _, _ in sets]
        for x in sets:
            x[2].random_(0, 256)
        torch.cuda.synchronize()
        for (cache, _, ws, mask, s, _), o in zip(sets, outs):
            rf.rf_attn_decode_paged_ex(cache, o, o, 0.0884, mask, ws, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
    for (cache, q, ws, mask, _, _), a in zip(sets, first):
        with pytest.raises(rf.RFError) as e:
            rf.rf_attn_decode_paged_ex(cache, q, a, 0.0884, mask, ws[:1024])
        assert e.value.status == rf.RF_ERR_WORKSPACE
    assert rf.rf_get_device_status() == rf.RF_OK


@pytest.mark.parametrize("kind,d,Tq", [(k, d, t) for k in ("e4m3", "bf16") for d in (64, 128)
                                       for t in (1, 3, 24)])
def test_pages_beyond_32_bits(rf, kind, d, Tq):  # noqa: F811
    """A pool of more than 2^31 elements a tensor; the sequences live in its last pages,
    a value that is not finite in front of the window."""
    num_pages, ps, e = 140000, 128, kind == "e4m3"
    bt = Batch(kind, [700, 310], 2, d, ps, seed=990)
    base = num_pages - bt.num_pages
    pages = [torch.zeros(num_pages, 2, ps, d, dtype=torch.uint8 if e else BF16, device="cuda")
             for _ in range(2)]
    scales = [torch.ones(num_pages, 2, device="cuda") if e else None for _ in range(2)]
    q = torch.randn(2, Tq, 8, d, generator=_gen(991)).to(BF16)
    ref, tol = masked_reference(q, bt, d ** -0.5, 150, 4)
    bt.pages[1][int(bt.table[0, 4]), 1, 8] = 0x7F if e else float("nan")        # key 520
    for t in range(2):
        pages[t][base:] = (torch.from_numpy(bt.pages[t]) if e else bt.pages[t]).cuda()
        if e:
            scales[t][base:] = torch.from_numpy(bt.scale[t]).cuda()
    cache = rf.rf_paged_kv(pages[0], pages[1], (bt.table + base).cuda(),
                           torch.tensor(bt.lens, dtype=torch.int32, device="cuda"), *scales)
    got, status = run(rf, bt, q, d ** -0.5, 150, 4, cache=cache)
    assert status == rf.RF_OK
    assert (np.abs(to64(got) - ref) <= tol).all()


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("G_", [128, 130])
def test_groups_of_a_whole_tile_and_more(rf, kind, G_):  # noqa: F811
    """More heads than a tile's 128 rows take the kernel with tiles of 16."""
    bt = Batch(kind, [200, 0, 33], 1, 64, 16, seed=995).garbage()
    for Tq, window, sinks, tree in ((1, 20, 3, False), (3, 0, 0, True)):
        q = torch.randn(3, Tq, G_, 64, generator=_gen(996)).to(BF16)
        M.check(rf, bt, q, 0.125, window, sinks, [tree_of(_gen(997), Tq)] * 3 if tree else None,
                f"{G_} heads")
