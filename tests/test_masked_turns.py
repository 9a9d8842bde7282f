"""The order in which the masked tensor-core kernel's warps wait for one another, walked
on the host: sequences whose last pair of query tiles is one tile, beside full pairs."""
import pytest
import torch


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    return m


# group, query tokens: 1 .. tpt tokens behind the full pairs of 2 tpt (tpt = 128 / group)
LAST_ALONE = [(8, 40), (8, 33), (8, 48), (5, 60), (1, 300), (16, 17), (128, 3)]


@pytest.mark.parametrize("G,Tq", LAST_ALONE)
@pytest.mark.parametrize("sms", [1, 3, 7, 152])
@pytest.mark.parametrize("tree", [0, 1])
def test_a_query_tiles_place_is_waited_for_in_turn(rf, G, Tq, sms, tree):
    lens = [Tq, 300, 0, Tq + 128, 3000, 2000, Tq, Tq + 1] * 2
    for window, sinks in ((0, 0), (100, 4)):
        assert rf.rf_selftest_masked_plan(torch.tensor(lens, dtype=torch.int32), None, None, len(lens), 2, G,
                                          Tq, 0, 4000, window, sinks, tree, sms) == 0
