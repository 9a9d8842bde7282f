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
