"""Paged-cache operators without a GPU: refusals through the C ABI, and the
library's own plans (work items of the append, partition of the decode) walked
on the host, with valid, ragged and inconsistent tables."""
import ctypes
import random

import pytest
import torch


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    return m


P = 1 << 20                       # a 16-byte aligned address, never dereferenced


def _cache(rf, **kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, block_table=P, seq_lens=P, dtype=rf.RF_E4M3, B=4,
             num_pages=100, page_size=64, max_pages=10, Hkv=2, d=128)
    d.update(kw)
    return rf._PagedKV(*[d[n] for n, _ in rf._PagedKV._fields_])


def _nr(rf, **kw):
    d = dict(cos=P, sin=P, max_pos=100, rot_dim=64, interleaved=0, q_weight=P, k_weight=P, eps=1e-6)
    d.update(kw)
    return rf._NormRope(*[d[n] for n, _ in rf._NormRope._fields_])


BAD_CACHE = [
    (dict(k=None), "arg"), (dict(v=P + 8), "arg"), (dict(block_table=None), "arg"),
    (dict(seq_lens=P + 2), "arg"), (dict(k_scale=None), "arg"), (dict(v_scale=P + 4), "arg"),
    (dict(dtype=0), "arg"), (dict(dtype=3), "arg"), (dict(B=0), "arg"), (dict(num_pages=0), "arg"),
    (dict(max_pages=0), "arg"), (dict(Hkv=-1), "arg"), (dict(page_size=0), "arg"),
    (dict(page_size=48), "unsupported"), (dict(page_size=256), "unsupported"),
    (dict(page_size=8), "unsupported"), (dict(d=96), "unsupported"), (dict(d=256), "unsupported"),
    (dict(num_pages=1 << 24, Hkv=2), "arg"), (dict(max_pages=(1 << 24) + 1), "arg"),
]


@pytest.mark.parametrize("bad,kind", BAD_CACHE)
def test_bad_caches_are_refused(rf, bad, kind):
    c = _cache(rf, **bad)
    want = rf.RF_ERR_INVALID_ARG if kind == "arg" else rf.RF_ERR_UNSUPPORTED
    assert rf.lib.rf_attn_decode_paged(c, P, P, 8, 1, 0.1, P, 1 << 30, None) == want
    assert rf.lib.rf_kv_append_paged(c, P, 256, P, 256, None, 4, None, None, 0, None, 0, 0,
                                     None) == want


def test_attn_decode_paged_refusals(rf):
    f, c = rf.lib.rf_attn_decode_paged, _cache(rf)
    big = 1 << 30
    for a in [(c, None, P, 8, 1, 0.1, P, big, None), (c, P, P + 4, 8, 1, 0.1, P, big, None),
              (c, P, P, 0, 1, 0.1, P, big, None), (c, P, P, 7, 1, 0.1, P, big, None),
              (c, P, P, 8, 0, 0.1, P, big, None), (c, P, P, 8, 1, 0.0, P, big, None),
              (c, P, P, 8, 1, -1.0, P, big, None), (c, P, P, 8, 1, float("nan"), P, big, None),
              (c, P, P, 8, 1, float("inf"), P, big, None), (c, P, P, 8, 1 << 28, 0.1, P, big, None),
              (_cache(rf, B=1 << 20, max_pages=1 << 14), P, P, 8, 1, 0.1, P, big, None),
              (None, P, P, 8, 1, 0.1, P, big, None)]:
        assert f(*a) == rf.RF_ERR_INVALID_ARG
    assert f(c, P, P, 8, 1, 0.1, None, big, None) == rf.RF_ERR_WORKSPACE
    assert f(c, P, P, 8, 1, 0.1, P + 4, big, None) == rf.RF_ERR_WORKSPACE
    for a in [(0, 8, 2, 1, 128), (1, 8, 3, 1, 128), (1, 8, 2, 0, 128), (1, 8, 2, 1, 96)]:
        assert rf.rf_attn_decode_paged_workspace_size(*a) == 0


def test_append_refusals(rf):
    c = _cache(rf)

    def call(c=c, K=P, ldk=256, V=P, ldv=256, cu=None, total=4, nr=None, Q=None, ldq=0, Qo=None,
             ldqo=0, Hq=0):
        return rf.lib.rf_kv_append_paged(c, K, ldk, V, ldv, cu, total, nr, Q, ldq, Qo, ldqo, Hq,
                                         None)

    for kw in [dict(K=None), dict(V=P + 8), dict(ldk=248), dict(ldv=257), dict(ldk=1 << 39),
               dict(total=0), dict(total=6), dict(total=-4), dict(cu=P + 2), dict(Hq=-1), dict(Hq=1),
               dict(Hq=2, Q=P, Qo=P, ldq=256, ldqo=128), dict(Hq=2, Q=P, Qo=None, ldq=256, ldqo=256),
               dict(Hq=1 << 20, total=1 << 16, Q=P, Qo=P, ldq=1 << 27, ldqo=1 << 27)]:
        assert call(**kw) == rf.RF_ERR_INVALID_ARG, kw
    for kw in BAD_NR:
        assert call(nr=_nr(rf, **kw)) == rf.RF_ERR_INVALID_ARG, kw


BAD_NR = [dict(cos=None), dict(sin=P + 4), dict(max_pos=0), dict(rot_dim=8), dict(rot_dim=40),
          dict(rot_dim=144), dict(rot_dim=0), dict(interleaved=2), dict(k_weight=P + 2),
          dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))]


def test_qk_norm_rope_refusals(rf):
    def call(dtype=1, Q=P, ldq=256, K=P, ldk=128, Qo=P, ldqo=256, Ko=P, ldko=128, pos=P, nr=None,
             T=4, Hq=2, Hkv=1, d=128):
        return rf.lib.rf_qk_norm_rope(dtype, Q, ldq, K, ldk, Qo, ldqo, Ko, ldko, pos, nr, T, Hq, Hkv,
                                      d, None)

    for kw in [dict(dtype=2), dict(dtype=-1), dict(Q=None), dict(Ko=P + 8), dict(ldq=128),
               dict(ldko=130), dict(T=0), dict(Hq=0, Hkv=0), dict(Hq=-1), dict(T=1 << 30, Hq=2),
               dict(nr=_nr(rf), pos=None), dict(nr=_nr(rf), pos=P + 1)]:
        assert call(**kw) == rf.RF_ERR_INVALID_ARG, kw
    for kw in BAD_NR:
        assert call(nr=_nr(rf, **kw)) == rf.RF_ERR_INVALID_ARG, kw
    assert call(d=96) == rf.RF_ERR_UNSUPPORTED
    assert call(d=256) == rf.RF_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors(rf):
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rf.rf_qk_norm_rope(x, None, x, None, None)
    with pytest.raises(ValueError):
        rf.rf_paged_kv(torch.zeros(1, 1, 16, 64, dtype=torch.uint8), None, None, None)
    with pytest.raises(ValueError):
        rf.rf_norm_rope(cos=torch.zeros(4, 8))


# ------------------------------------------------------------------ plans


def _table(rng, B, max_pages, num_pages, lens, ps, bad=0.0):
    t = torch.randint(-5, 3 * num_pages, (B, max_pages), dtype=torch.int32)   # unused: anything
    for b in range(B):
        n = max(0, -(-lens[b] // ps))
        for i in range(min(n, max_pages)):
            t[b, i] = rng.randrange(num_pages) if rng.random() >= bad else rng.choice(
                [-1, num_pages, 2**31 - 1, -2**31])
    return t


@pytest.mark.parametrize("seed", range(60))
def test_append_plan(rf, seed):
    rng = random.Random(seed)
    B, ps = rng.choice([1, 2, 3, 7, 33, 100]), rng.choice([16, 32, 64, 128])
    max_pages = rng.randint(1, 12)
    cap = max_pages * ps
    uniform = rng.random() < 0.4
    if uniform:
        n = rng.choice([1, 1, 2, ps - 1, ps, ps + 1, cap])
        new = [min(n, cap)] * B
    else:
        new = [rng.choice([0, 0, 1, 2, rng.randint(0, cap), ps, cap]) for _ in range(B)]
        new[rng.randrange(B)] = rng.randint(1, cap)
    lens = [min(cap, m + rng.choice([0, 1, ps - 1, ps, rng.randint(0, cap)])) for m in new]
    if seed % 3 == 0:                                       # padded rows
        lens = [0 if rng.random() < 0.3 else n for n in lens]
    max_pos = 0
    if seed % 4 == 1:                                       # inconsistent lengths
        lens[rng.randrange(B)] = rng.choice([-1, cap + 1, 2**31 - 1, -2**31])
        max_pos = rng.randint(1, cap)
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
    table = _table(rng, B, max_pages, 50, lens, ps, bad=0.2 if seed % 5 == 2 else 0.0)
    assert rf.rf_selftest_append_plan(table, torch.tensor(lens, dtype=torch.int32),
                                      None if uniform else cu, sum(new), 50, ps, max_pos) == 0


@pytest.mark.parametrize("seed", range(40))
def test_append_plan_stays_in_bounds_with_disordered_cu_seqlens(rf, seed):
    rng = random.Random(1000 + seed)
    B, ps, total = rng.randint(1, 40), rng.choice([16, 64]), rng.randint(1, 500)
    cu = torch.tensor([rng.choice([rng.randint(-3, total + 3), -2**31, 2**31 - 1, 0, total])
                       for _ in range(B + 1)], dtype=torch.int32)
    lens = torch.tensor([rng.randint(0, 8 * ps) for _ in range(B)], dtype=torch.int32)
    table = _table(rng, B, 8, 20, lens.tolist(), ps)
    assert rf.rf_selftest_append_plan(table, lens, cu, total, 20, ps, 0) == 0


@pytest.mark.parametrize("between,tokens", [(1, 100), (41, 2000)])
def test_append_plan_with_items_of_several_sequences(rf, between, tokens):
    """Two sequences claim the same items: each claim stays in bounds."""
    cu = torch.tensor([0] + [tokens] * between + [0, tokens], dtype=torch.int32)
    B, pages = between + 2, -(-tokens // 16)
    lens = torch.tensor([tokens] + [0] * between + [tokens], dtype=torch.int32)
    table = torch.arange(B * pages, dtype=torch.int32).view(B, pages)
    assert rf.rf_selftest_append_plan(table, lens, cu, tokens, B * pages, 16, 0) == 0


@pytest.mark.parametrize("seed", range(80))
def test_decode_plan(rf, seed):
    rng = random.Random(seed)
    B = rng.choice([1, 1, 2, 5, 32, 33, 200, 700])
    top = rng.choice([1, 40, 500, 9000 if B < 50 else 700])
    lens = [rng.choice([0, 1, 31, 32, 33, rng.randint(0, top), top]) for _ in range(B)]
    if seed % 5 == 0:
        lens[rng.randrange(B)] = rng.choice([-1, -2**31, 2**31 - 1, 20000])   # count as empty
    t = torch.tensor(lens, dtype=torch.int32)
    for warps in (4, 8):
        assert rf.rf_selftest_decode_paged_plan(t, rng.choice([1, 2, 7, 8]), 10000, warps,
                                                rng.choice([1, 3, 148, 152])) == 0


def test_decode_plan_of_a_long_context(rf):
    t = torch.tensor([2**30, 5, 2**29 + 1], dtype=torch.int32)     # 2^30 chunks over 8 tiles at most
    assert rf.rf_selftest_decode_paged_plan(t[1:], 1, 2**30, 8, 152) == 0
    assert rf.rf_selftest_decode_paged_plan(t, 64, 2**30, 8, 152) == -1


def test_plans_refuse_bad_sizes(rf):
    t = torch.ones(2, dtype=torch.int32)
    for a in [(0, 100, 8, 152), (1, 0, 8, 152), (1, 100, 5, 152), (1, 100, 8, 0)]:
        assert rf.rf_selftest_decode_paged_plan(t, *a) == -1
    table = torch.zeros(2, 3, dtype=torch.int32)
    assert rf.rf_selftest_append_plan(table, t, None, 3, 10, 16) == -1
    assert rf.rf_selftest_append_plan(table, t, None, 2, 0, 16) == -1
    assert rf.lib.rf_selftest_append_plan(None, ctypes.c_void_p(t.data_ptr()), None, 2, 2, 10, 16,
                                          3, 0) == -1
