"""Values at which the paged-cache operators can go wrong: zeros with a sign,
products of fp32 range, and attention rows whose weights span many binades.
Tolerances count half steps of rounding, as in test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from oracle import paged as G
from tests.helpers import to64
from tests.test_gpu_paged import BF16, F32, NR, Batch, _gen, _tables, assert_rows

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
