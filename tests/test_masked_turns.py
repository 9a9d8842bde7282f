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


# more new tokens than keys: query tiles and whole sequences that read nothing
NO_KEYS = [([300, 1, 128, 129, 40, 300], [0, 1, 0, 10, 0, 300]), ([700], [3]),
           ([500, 20, 20, 20, 900], [90, 0, 0, 0, 0])]


@pytest.mark.parametrize("new,keys", NO_KEYS)
@pytest.mark.parametrize("G", [1, 4, 5, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (16, 2), (2**30, 200)])
def test_a_prompts_tiles_all_have_scores(rf, new, keys, G, window, sinks):
    cu = [torch.tensor([0] + x, dtype=torch.int32).cumsum(0).to(torch.int32) for x in (new, keys)]
    for sms in (1, 3, 152):
        assert rf.rf_selftest_masked_plan(None, cu[0], cu[1], len(new), 2, G, max(new), sum(new), sum(keys),
                                          window, sinks, 0, sms) == 0
