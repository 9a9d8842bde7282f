"""Masked attention without a GPU: refusals through the C ABI, and the decode's plan
with windows walked on the host."""
import random

import pytest
import torch

from tests.test_paged_host import BAD_CACHE, P, _cache


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    return m


def _mask(rf, window=0, sinks=0, parents=None):
    return rf._AttnMask(window, sinks, parents)


@pytest.mark.parametrize("bad,kind", BAD_CACHE)
def test_bad_caches_are_refused(rf, bad, kind):
    want = rf.RF_ERR_INVALID_ARG if kind == "arg" else rf.RF_ERR_UNSUPPORTED
    assert rf.lib.rf_attn_decode_paged_ex(_cache(rf, **bad), P, P, 8, 1, 0.1, _mask(rf, 5), P, 1 << 30,
                                          None) == want


def test_attn_decode_paged_ex_refusals(rf):
    f, c, big = rf.lib.rf_attn_decode_paged_ex, _cache(rf), 1 << 30
    for m in (_mask(rf, -1), _mask(rf, 5, -1), _mask(rf, (1 << 30) + 1), _mask(rf, 5, (1 << 30) + 1),
              _mask(rf, 0, 0, P + 2)):
        assert f(c, P, P, 8, 1, 0.1, m, P, big, None) == rf.RF_ERR_INVALID_ARG
    for m in (None, _mask(rf, 5, 2), _mask(rf, 0, 0, P)):
        for a in [(None, P, 8, 1, 0.1), (P, P + 4, 8, 1, 0.1), (P, P, 0, 1, 0.1), (P, P, 7, 1, 0.1),
                  (P, P, 8, 0, 0.1), (P, P, 8, 1, 0.0), (P, P, 8, 1, float("nan")),
                  (P, P, 8, 1 << 28, 0.1)]:
            assert f(c, *a, m, P, big, None) == rf.RF_ERR_INVALID_ARG
        assert f(None, P, P, 8, 1, 0.1, m, P, big, None) == rf.RF_ERR_INVALID_ARG
        assert f(c, P, P, 8, 1, 0.1, m, None, big, None) == rf.RF_ERR_WORKSPACE
        assert f(c, P, P, 8, 1, 0.1, m, P + 4, big, None) == rf.RF_ERR_WORKSPACE
    tree = _mask(rf, 0, 0, P)
    assert f(c, P, P, 8, 4097, 0.1, tree, P, big, None) == rf.RF_ERR_INVALID_ARG
    assert f(c, P, P, 8, 4096, 0.1, tree, None, big, None) == rf.RF_ERR_WORKSPACE
    for a in [(0, 8, 2, 1, 128), (1, 8, 3, 1, 128), (1, 8, 2, 0, 128), (1, 8, 2, 1, 96)]:
        assert rf.rf_attn_decode_paged_ex_workspace_size(*a) == 0


def test_binding_refuses_bad_masks(rf):
    for a in [(-1,), (5, -1), (2**30 + 1,), (0, 0, torch.zeros(1, 3, dtype=torch.int32))]:
        with pytest.raises(ValueError):
            rf.rf_attn_mask(*a)


@pytest.mark.parametrize("seed", range(120))
def test_decode_plan_with_a_window(rf, seed):
    rng = random.Random(seed)
    B = rng.choice([1, 1, 2, 5, 32, 33, 200])
    top = rng.choice([1, 40, 500, 9000])
    lens = [rng.choice([0, 1, 31, 32, 33, rng.randint(0, top), top]) for _ in range(B)]
    if seed % 5 == 0:
        lens[rng.randrange(B)] = rng.choice([-1, -2**31, 2**31 - 1, 20000])   # count as empty
    t = torch.tensor(lens, dtype=torch.int32)
    window = rng.choice([1, 31, 32, 33, rng.randint(1, top), 2**30])
    sinks = rng.choice([0, 1, 4, 32, 33, rng.randint(0, top), 2**30])
    Tq = rng.choice([1, 1, 2, 40, 2 * top])
    for warps in (4, 8):
        assert rf.rf_selftest_decode_paged_ex_plan(t, rng.choice([1, 2, 7]), 10000, Tq, window, sinks, warps,
                                                   rng.choice([1, 3, 148, 152])) == 0


def test_plan_refuses_bad_sizes(rf):
    t = torch.ones(2, dtype=torch.int32)
    for a in [(1, 100, 0, 5, 0, 8, 152), (1, 100, 1, 0, 0, 8, 152), (1, 100, 1, -1, 0, 8, 152),
              (1, 100, 1, 5, -1, 8, 152), (1, 100, 1, 5, 0, 5, 152), (0, 100, 1, 5, 0, 8, 152)]:
        assert rf.rf_selftest_decode_paged_ex_plan(t, *a) == -1


# ------------------------------------------------------------------ prompts and many rows


def test_attn_fwd_window_refusals(rf):
    def call(Q=P, ldq=512, K=P, ldk=256, V=P, ldv=256, O=P, ldo=512, cq=P, ck=P, B=2, Hq=4, Hkv=2, mq=60,
             tq=100, tk=120, d=128, scale=0.1, window=16, sinks=4):
        return rf.lib.rf_attn_fwd_window(Q, ldq, K, ldk, V, ldv, O, ldo, cq, ck, B, Hq, Hkv, mq, tq, tk, d,
                                         scale, window, sinks, None)

    for kw in [dict(Q=None), dict(K=P + 8), dict(V=None), dict(O=P + 4), dict(cq=P + 2), dict(ck=P + 1),
               dict(ldq=504), dict(ldk=260), dict(ldv=128), dict(ldo=516), dict(ldq=1 << 39, tq=1, mq=1),
               dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(mq=0), dict(mq=101), dict(tq=0),
               dict(tk=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(window=(1 << 30) + 1),
               dict(sinks=(1 << 30) + 1), dict(cq=None, tq=101, mq=60), dict(cq=None, mq=49),
               dict(ck=None, tk=121), dict(tq=(1 << 30) + 1), dict(tk=(1 << 30) + 1),
               dict(B=1 << 25, mq=100), dict(Hq=1 << 21, ldq=1 << 29, ldo=1 << 29, Hkv=1 << 20)]:
        assert call(**kw) == rf.RF_ERR_INVALID_ARG, kw
    assert call(d=96) == rf.RF_ERR_UNSUPPORTED
    assert call(Hq=258, ldq=258 * 128, ldo=258 * 128, Hkv=2) == rf.RF_ERR_UNSUPPORTED


@pytest.mark.parametrize("seed", range(150))
def test_plan_of_prompts(rf, seed):
    rng = random.Random(seed)
    B, Hkv = rng.choice([1, 1, 2, 5, 20]), rng.choice([1, 2, 3, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 31, 64, 100, 128])
    top = rng.choice([1, 3, 130, 600])
    new = [rng.choice([0, 1, rng.randint(0, top), top]) for _ in range(B)]
    new[rng.randrange(B)] = top
    keys = [max(0, n + rng.choice([0, 0, 1, -1, rng.randint(0, 400), -n])) for n in new]
    keys[rng.randrange(B)] += 1
    mq = rng.choice([max(new), sum(new)])
    window = rng.choice([0, 1, 2, 127, 128, 129, rng.randint(1, 700), 2**30])
    sinks = rng.choice([0, 1, 4, 128, 129, rng.randint(0, 700), 2**30])
    cu = [torch.tensor([0] + x, dtype=torch.int32).cumsum(0).to(torch.int32) for x in (new, keys)]
    if seed % 6 == 0:                                       # out of order, too long
        cu[rng.randrange(2)][rng.randrange(B + 1)] = rng.choice([-1, 2**31 - 1, -2**31, 0, 10**6])
    assert rf.rf_selftest_masked_plan(None, cu[0], cu[1], B, Hkv, G, mq, sum(new), sum(keys), window, sinks,
                                      0, rng.choice([1, 3, 148, 152])) == 0


@pytest.mark.parametrize("seed", range(150))
def test_plan_of_many_rows_over_a_cache(rf, seed):
    rng = random.Random(500 + seed)
    B, Hkv = rng.choice([1, 1, 2, 5, 12]), rng.choice([1, 2, 3, 8])
    G, Tq = rng.choice([1, 2, 3, 4, 5, 8, 16, 128]), rng.choice([1, 2, 7, 25, 64, 200])
    top = rng.choice([1, 40, 500, 3000])
    lens = [rng.choice([0, 1, 127, 128, 129, rng.randint(0, top), top, Tq, max(0, Tq - 1)]) for _ in range(B)]
    lens = [min(n, 4000) for n in lens]
    if seed % 5 == 0:
        lens[rng.randrange(B)] = rng.choice([-1, -2**31, 2**31 - 1, 20000])   # count as empty
    window = rng.choice([0, 1, 128, rng.randint(1, 700), 2**30])
    sinks = rng.choice([0, 1, 4, 129, rng.randint(0, 700)])
    assert rf.rf_selftest_masked_plan(torch.tensor(lens, dtype=torch.int32), None, None, B, Hkv, G, Tq, 0,
                                      4000, window, sinks, rng.randint(0, 1),
                                      rng.choice([1, 3, 148, 152])) == 0


def test_masked_plan_refuses_bad_sizes(rf):
    t = torch.ones(2, dtype=torch.int32)
    good = [t, None, None, 2, 1, 4, 8, 0, 100, 5, 0, 0, 152]
    assert rf.rf_selftest_masked_plan(*good) == 0
    for i, x in ((4, 0), (5, 0), (5, 129), (6, 0), (8, 0), (9, -1), (10, -1), (11, 2), (12, 0)):
        bad = list(good)
        bad[i] = x
        assert rf.rf_selftest_masked_plan(*bad) == -1
    assert rf.rf_selftest_masked_plan(None, None, None, 2, 1, 4, 8, 15, 100, 5, 0, 0, 152) == -1
    assert rf.rf_selftest_masked_plan(None, None, None, 2, 1, 4, 8, 16, 100, 5, 0, 1, 152) == -1
