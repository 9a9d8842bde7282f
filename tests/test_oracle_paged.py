"""Pins of the paged-cache oracle (CPU): closed forms, library routines and
identities."""
import numpy as np
import pytest
import torch

from oracle import paged as G
from oracle.fp8_quant_gemm import e4m3_decode, e4m3_encode


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def _tables(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None, :]
    return np.cos(a), np.sin(a)


def test_rotation_is_a_complex_product():
    x = _rand(1, 5, 3, 16)
    cos, sin = _tables(40, 16)
    pos = np.array([0, 7, 39, 7, 1])
    z = (cos + 1j * sin)[pos][:, None, :]
    y = G.norm_rope(x, pos, cos, sin)
    got = y[..., :8] + 1j * y[..., 8:]
    np.testing.assert_allclose(got, (x[..., :8] + 1j * x[..., 8:]) * z, atol=1e-14)
    y = G.norm_rope(x, pos, cos, sin, interleaved=True)
    np.testing.assert_allclose(y[..., ::2] + 1j * y[..., 1::2], (x[..., ::2] + 1j * x[..., 1::2]) * z,
                               atol=1e-14)


def test_scores_depend_on_the_distance_only():
    cos, sin = _tables(100, 32)
    q, k = _rand(2, 1, 1, 32), _rand(3, 1, 1, 32)
    dot = [float((G.norm_rope(q, [p + 9], cos, sin) * G.norm_rope(k, [p], cos, sin)).sum())
           for p in (0, 13, 90)]
    np.testing.assert_allclose(dot, dot[0], rtol=1e-12)


def test_partial_rotation_leaves_the_rest():
    x = _rand(4, 3, 2, 64)
    cos, sin = _tables(10, 16)
    y = G.norm_rope(x, [1, 2, 3], cos, sin)
    assert (y[..., 16:] == x[..., 16:]).all() and (y[..., :16] != x[..., :16]).all()


def test_norm_matches_the_library():
    x, w = _rand(5, 4, 3, 64), _rand(6, 64)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-6)
    np.testing.assert_allclose(G.norm_rope(x, None, weight=w), ref.numpy(), rtol=1e-12)


@pytest.mark.parametrize("a,s", [(448.0, 1.0), (448.0000001, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                 (1.7500001, 2.0 ** -7), (0.0, 2.0 ** -126), (3e38, 2.0 ** 120)])
def test_pow2_scale(a, s):
    assert G.pow2_scale(a) == s


def test_rescaled_codes_stand_for_the_same_values():
    codes = e4m3_encode(_rand(7, 16, 64) * 50)
    codes[5:] = 0
    x = np.full((1, 64), 3.0)
    x[0, 0] = 448.0 * 4
    new, s = G.append_e4m3(codes, 0.5, x, 5)
    assert s == 4.0
    was, now = e4m3_decode(codes[:5]) * 0.5, e4m3_decode(new[:5]) * s
    normal = np.abs(was) >= 4 * 2.0 ** -6
    assert (was[normal] == now[normal]).all()                # exact but for subnormals
    assert np.abs(was - now).max() <= 4 * 2.0 ** -10
    assert (e4m3_decode(new[5]) * s == np.where(x[0] == 3.0, 3.0, 1792.0)).all()
    assert (new[6:] == codes[6:]).all()


def test_a_page_begun_anew_forgets_its_scale():
    codes = np.full((16, 64), 0x7F, np.uint8)
    new, s = G.append_e4m3(codes, 1e30, np.ones((2, 64)), 0)
    assert s == 2.0 ** -8 and (e4m3_decode(new[:2]) * s == 1).all() and (new[2:] == 0x7F).all()


def test_infinities_saturate_and_nan_stays():
    x = np.ones((1, 4))
    x[0, 1:] = [np.inf, -np.inf, np.nan]
    new, s = G.append_e4m3(np.zeros((16, 4), np.uint8), 1.0, x, 0)
    assert s == 2.0 ** -8 and list(new[0]) == [0x78, 0x7E, 0xFE, 0x7F]


def test_token_by_token_equals_a_chunk_where_rescaling_is_exact():
    rng = np.random.default_rng(8)
    k = np.exp2(rng.integers(-3, 4, (40, 2, 64)))            # no code becomes subnormal
    v = -k
    table = np.array([[2, 0, 1]])

    def empty():
        return [np.zeros((3, 2, 16, 64), np.uint8)] * 2 + [np.ones((3, 2), np.float32)] * 2

    whole = G.append(*empty(), table, [40], [40], k, v)
    state = empty()
    for t in range(40):
        state = G.append(*state, table, [t + 1], [1], k[t:t + 1], v[t:t + 1])
    for a, b in zip(whole, state):
        np.testing.assert_array_equal(a, b)


def test_decode_matches_library_attention():
    B, Tq, Hq, Hkv, d, ps, n = 2, 3, 4, 2, 16, 16, 37
    K, V = _rand(9, 7, Hkv, ps, d), _rand(10, 7, Hkv, ps, d)
    q = _rand(11, B, Tq, Hq, d)
    table = np.array([[3, 1, 6], [0, 4, 2]])
    o = G.decode(q, K, V, None, None, table, [n, n], 0.3)
    for b in range(B):
        kb = K[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n].repeat(Hq // Hkv, 0)
        vb = V[table[b]].transpose(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :n].repeat(Hq // Hkv, 0)
        mask = torch.arange(n)[None, :] <= torch.arange(n - Tq, n)[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[b].transpose(1, 0, 2)), torch.from_numpy(kb), torch.from_numpy(vb),
            attn_mask=mask, scale=0.3)
        np.testing.assert_allclose(o[b], ref.numpy().transpose(1, 0, 2), atol=1e-13)


def test_rows_without_keys_are_zero():
    K = _rand(12, 1, 1, 16, 8)
    o = G.decode(_rand(13, 2, 4, 1, 8), K, K, None, None, [[0], [0]], [2, 0], 1.0)
    assert (o[0, :2] == 0).all() and (o[1] == 0).all() and (o[0, 2, 0] == K[0, 0, 0]).all()
