"""Values at which the paged-cache operators can go wrong: zeros with a sign,
products of fp32 range, and attention rows whose weights span many binades.
Tolerances count half steps of rounding, as in test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from oracle import paged as G
from oracle.fp8_quant_gemm import e4m3_encode
from tests.helpers import to64
from tests.test_gpu_paged import BF16, F32, NR, Batch, _gen, _tables, assert_rows, attn_reference, \
    check_attn, run_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    assert torch.cuda.is_available()
    assert m.rf_get_device_status() == m.RF_OK
    return m


def _bits(t):
    return t.cpu().contiguous().view(torch.int32 if t.dtype == F32 else torch.int16)


# ------------------------------------------------------------------ norm and rotation


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_copy_keeps_the_sign_of_zeros(rf, dtype, d):
    x = torch.randn(9, 5, d, generator=_gen(d)).to(dtype)
    x[torch.rand(9, 5, d, generator=_gen(d + 1)) < 0.3] = -0.0
    x[torch.rand(9, 5, d, generator=_gen(d + 2)) < 0.2] = 0.0
    o = torch.empty_like(x, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), None, o, None, None)
    assert torch.equal(_bits(o), _bits(x))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_elements_behind_the_rotation_keep_the_sign_of_zeros(rf, inter, norm):
    """Of the weights' signs, too, where there is a norm."""
    nr = NR(rf, 128, 64, inter, norm, BF16)
    if norm:
        nr.w["q"][::3] *= -1
        nr.dev.q_weight.copy_(nr.w["q"])
    x = torch.randn(7, 2, 128, generator=_gen(3)).to(BF16)
    x[..., 64:][torch.rand(7, 2, 64, generator=_gen(4)) < 0.4] = -0.0
    pos = torch.arange(7, dtype=torch.int32)
    o = torch.empty_like(x, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), None, o, None, nr.dev, pos.cuda())
    ref = nr.ref(x, pos, "q")
    assert_rows(o, ref, BF16, "q")
    np.testing.assert_array_equal(np.signbit(to64(o))[..., 64:], np.signbit(ref)[..., 64:])


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("new", [1, 4, 40])
def test_unrotated_append_keeps_the_sign_of_zeros(rf, kind, new):
    bt = Batch(kind, [new], 2, 64, 16, seed=5)
    cache = bt.device(rf)
    k, v = (torch.randn(new, 2, 64, generator=_gen(6 + i)).to(BF16) for i in range(2))
    for t in (k, v):
        t[torch.rand(new, 2, 64, generator=_gen(8)) < 0.3] = -0.0
    rf.rf_kv_append_paged(cache, k.cuda(), v.cuda())
    for t, got in ((k, bt.k.t), (v, bt.v.t)):
        g = got.cpu()[bt.table[0, :-(-new // 16)].long()].transpose(1, 2).reshape(-1, 2, 64)[:new]
        sign = (g >= 0x80).numpy() if kind == "e4m3" else np.signbit(to64(g))
        np.testing.assert_array_equal(sign, np.signbit(to64(t)))


def test_an_infinite_weight_spoils_its_own_element_only(rf):
    """Behind the rotation, where elements have no partner."""
    w = torch.ones(128, dtype=BF16)
    w[100] = float("inf")
    cos, sin = _tables(16, 64)
    for inter in (False, True):
        nr = rf.rf_norm_rope(cos.cuda(), sin.cuda(), inter, w.cuda(), None, 1e-6)
        x = torch.randn(5, 3, 128, generator=_gen(9)).to(BF16)
        pos = torch.arange(5, dtype=torch.int32)
        o = torch.empty_like(x, device="cuda")
        rf.rf_qk_norm_rope(x.cuda(), None, o, None, nr, pos.cuda())
        got, finite = to64(o), [i for i in range(128) if i != 100]
        ref = G.norm_rope(x, pos, cos, sin, inter, torch.ones(128, dtype=BF16))
        assert_rows(got[..., finite], ref[..., finite], BF16, "finite elements")
        assert np.isinf(got[..., 100]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("x_exp,w_exp", [(50, 100), (-50, -100), (60, 120)])
def test_norm_comes_before_the_weight(rf, dtype, inter, x_exp, w_exp):
    """x * w leaves fp32's range where the normed row times w does not."""
    cos, sin = _tables(40, 32)
    w = ((1 + 0.3 * torch.rand(64, generator=_gen(10))) * 2.0 ** w_exp).to(dtype)
    x = (torch.randn(33, 3, 64, generator=_gen(11)) * 2.0 ** x_exp).to(dtype)
    pos = torch.arange(33, dtype=torch.int32)
    nr = rf.rf_norm_rope(cos.cuda(), sin.cuda(), inter, w.cuda(), None, 2.0 ** -120)
    o = torch.empty_like(x, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), None, o, None, nr, pos.cuda())
    ref = G.norm_rope(x, pos, cos, sin, inter, w, 2.0 ** -120)
    assert_rows(to64(o) * 2.0 ** -w_exp, ref * 2.0 ** -w_exp, dtype, "normed rows")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_whose_mean_of_squares_is_infinite_become_zeros(rf, dtype):
    nr = NR(rf, 64, 64, False, True, dtype)
    x = (torch.randn(5, 2, 64, generator=_gen(12)) * 2.0 ** 70).to(dtype)
    x[3] = torch.finfo(dtype).max
    x[4] = torch.randn(2, 64, generator=_gen(13)).to(dtype)
    pos = torch.arange(5, dtype=torch.int32)
    o = torch.empty_like(x, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), None, o, None, nr.dev, pos.cuda())
    assert (o[:4] == 0).all()
    assert_rows(o[4:], nr.ref(x[4:], pos[4:], "q"), dtype, "the other rows")


# ------------------------------------------------------------------ weights of many binades


def _sink(kind, n, d, gap, first, seed, G_, Tq):
    """Sequences of the same n keys, more of them than the device has warps, so that
    a warp streams whole ones: the first key's score is `gap` nats above every
    other one's (to within the others' own spread, about 0.05 sqrt(d)), and the
    values of its chunk of 32 keys are `first` times the others'."""
    bt = Batch(kind, [n], 1, d, 64, seed=seed, loud=0.0)
    g = _gen(seed + 1)
    x = 0.05 * torch.randn(2, bt.num_pages, 1, 64, d, generator=g)
    x[1] *= 20
    x[0, ..., 0] = 0
    p0 = int(bt.table[0, 0])
    x[0, p0, 0, 0] = 0
    x[0, p0, 0, 0, 0] = 0.25
    x[1, p0, 0, :32] *= first
    if kind == "e4m3":
        bt.scale[0], bt.scale[1] = 2.0 ** -10, 2.0 ** -7
        bt.pages = e4m3_encode(x.numpy() / bt.scale[..., None, None])
    else:
        bt.pages = x.to(BF16)
    q = torch.randn(1, Tq, G_, d, generator=g).to(BF16)
    q[..., 0] = 4 * gap
    return bt, q


def _weighted(bt, q, scale):
    """(o, tolerance) of one sequence and kv head: fp64, and the half steps of the
    output (2^-8), of a weight (2^-11 relative in f16) and of the scores (d products
    and sums in fp32, the exponential's argument and result).  A weight below f16's
    normal numbers is off by 2^-25 of what is 2^15 for the sequence's first chunk's
    largest, and 2^-1 at least for a later chunk's."""
    qq = to64(q)[0]
    n, ps, d = bt.lens[0], bt.ps, bt.d
    pages = bt.table[0, :-(-n // ps)].numpy()
    K, V = (G.values(*bt.host(i))[pages, 0].reshape(-1, d)[:n] for i in (0, 1))
    Tq = len(qq)
    o, tol = np.zeros_like(qq), np.zeros_like(qq)
    for t in range(Tq):
        m = n - Tq + t + 1
        s = scale * qq[t] @ K[:m].T
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        size = scale * np.abs(qq[t]) @ np.abs(K[:m]).T
        u = 2.0 ** -23
        per = 2 * ((d + 8) * u * size.max(1) + 4 * u * np.abs(s).max(1) + 8 * u) + \
            2.0 ** -11 + (m / 8 + 64) * u
        small = np.repeat(np.stack([p[:, i:i + 32].max(1) * 2.0 ** (-24 if i else -40)
                                    for i in range(0, m, 32)], 1), 32, 1)[:, :m]
        o[t] = p @ V[:m]
        tol[t] = per[:, None] * (p @ np.abs(V[:m])) + small @ np.abs(V[:m])
    return o, tol + 2.0 ** -8 * (np.abs(o) + tol) + 1e-37


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("gap", [4, 10, 14, 16, 18, 22, 26, 30, 36])
@pytest.mark.parametrize("first", [0.0, 2.0 ** -7, 1.0])
@pytest.mark.parametrize("n,d,G_,Tq", [(2048, 128, 4, 1), (700, 64, 3, 4), (1000, 128, 12, 1)])
def test_a_dominant_key_does_not_drown_the_others(rf, kind, gap, first, n, d, G_, Tq):
    """The others' weights are e^-gap of the first key's, whose value is zero or
    small: their sum is all, or most, of the output."""
    bt, q = _sink(kind, n, d, gap, first, 800 + gap, G_, Tq)
    ref, tol = _weighted(bt, q, 1.0)
    warps = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    B = warps + warps // 16                   # the sequences' borders fall anywhere in a warp's range
    bt.lens, bt.table, bt.B = [n] * B, bt.table.expand(B, -1).contiguous(), B
    got, status = run_attn(rf, bt, q.expand(B, -1, -1, -1).contiguous(), 1.0)
    assert status == rf.RF_OK
    err = np.abs(to64(got) - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max():.2f} of the tolerance, " \
        f"{(np.linalg.norm(err, axis=(1, 2, 3)) / np.linalg.norm(ref)).max():.2e} relative"


@pytest.mark.parametrize("v_exp", [-114, -105, 112])
@pytest.mark.parametrize("lens", [[70, 5], [9000, 3]])
def test_value_scales_next_to_fp32s_ends(rf, v_exp, lens):
    """2^(M - m) alone, or its product with o, would leave fp32's range."""
    bt = Batch("e4m3", lens, 1, 128, 32, seed=830, loud=0.0)
    bt.scale[1] *= np.float32(2.0 ** v_exp)
    q = torch.randn(2, 1, 4, 128, generator=_gen(831)).to(BF16)
    check_attn(rf, bt, q, 128 ** -0.5, f"value scales of 2^{v_exp}")


@pytest.mark.parametrize("Tq,G_", [(1, 4), (4, 3)])
@pytest.mark.parametrize("exp", [4, 10, 16])
def test_scores_up_to_a_million(rf, Tq, G_, exp):
    """The largest weight's exponent is rounded by more than f16 has left above it."""
    bt = Batch("e4m3", [500, 33], 1, 64, 16, seed=832)
    q = (torch.randn(2, Tq, G_, 64, generator=_gen(833)) * 2.0 ** exp).to(BF16)
    got, status = run_attn(rf, bt, q, 1.0)
    assert status == rf.RF_OK
    ref, tol = attn_reference(q, bt, 1.0)
    assert (np.abs(to64(got) - ref) <= tol).all()
