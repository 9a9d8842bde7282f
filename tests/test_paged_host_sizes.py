"""The paged-cache operators' host code at sizes where a walk takes long or an
int ends."""
import pytest
import torch

from tests.test_paged_host import P, _cache


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    return m


@pytest.mark.parametrize("use_cu", [False, True])
def test_append_plan_of_the_largest_batch_is_walked_in_seconds(rf, use_cu):
    B = 1 << 20
    table = torch.arange(B, dtype=torch.int32)[:, None]
    lens = torch.ones(B, dtype=torch.int32)
    cu = torch.arange(B + 1, dtype=torch.int32) if use_cu else None
    assert rf.rf_selftest_append_plan(table, lens, cu, B, B, 16) == 0
    table[B // 3] = -1                          # noticed, and no other check fails
    assert rf.rf_selftest_append_plan(table, lens, cu, B, B, 16) == 0


def test_append_plan_of_a_large_disordered_batch_is_refused_at_once(rf):
    """Every second sequence claims every token: 2^17 times 2^20 items."""
    B, total = 1 << 18, 1 << 24
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1::2] = total
    table = torch.zeros(B, 1, dtype=torch.int32)
    lens = torch.ones(B, dtype=torch.int32)
    assert rf.rf_selftest_append_plan(table, lens, cu, total, 1, 16) == -1


def test_attn_of_nearly_2_31_rows(rf):
    """Tq * Hq / Hkv up to 2^31 - 1: the tiles of a kv head are counted without
    overflow, so that 2^27 of them with 20 chunks of keys each are refused; sizes
    just within the limits come as far as the workspace."""
    def call(Hq, Tq, **kw):
        return rf.lib.rf_attn_decode_paged(_cache(rf, B=1, Hkv=1, **kw), P, P, Hq, Tq, 0.1, None, 0,
                                           None)

    for Hq, Tq in [(2**31 - 1, 1), (2**31 - 16, 1), (2**31 - 17, 1), ((2**31 - 1) // 3, 3),
                   (1, 2**31 - 1), ((2**31 - 1) // 7, 7)]:
        assert call(Hq, Tq) == rf.RF_ERR_INVALID_ARG, (Hq, Tq)
        assert call(Hq, Tq, max_pages=7) == rf.RF_ERR_WORKSPACE, (Hq, Tq)      # 14 chunks
    for Hq, Tq in [(2**30, 2), ((2**31 - 1) // 3 + 1, 3)]:
        assert call(Hq, Tq, max_pages=1) == rf.RF_ERR_INVALID_ARG, (Hq, Tq)
