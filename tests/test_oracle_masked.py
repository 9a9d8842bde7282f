"""Oracle of the masked attention (windows with sinks, trees of drafted tokens)
against a library routine with explicit masks, closed forms and worked examples."""
import numpy as np
import pytest
import torch

from oracle import paged as G


def test_seen_keys_worked_examples():
    # 10 tokens, the last two query; window 3 of position 8: 6 7 8; of 9: 7 8 9
    assert G.seen_keys(10, 2, 0, 3, 0) == [6, 7, 8]
    assert G.seen_keys(10, 2, 1, 3, 2) == [0, 1, 7, 8, 9]
    assert G.seen_keys(10, 2, 1, 3, 8) == list(range(10))        # sinks up to the window
    assert G.seen_keys(3, 1, 0, 100, 4) == [0, 1, 2]
    assert G.seen_keys(10, 1, 0, 1, 0) == [9]
    assert G.seen_keys(2, 4, 0) == G.seen_keys(2, 4, 1) == []    # rows before the sequence
    assert G.seen_keys(2, 4, 2) == [0]
    # 5 tokens and a tree: 0 - 1 - 3, 0 - 2, and a second root 4
    tree = [-1, 0, 0, 1, -1]
    assert G.seen_keys(10, 5, 0, parents=tree) == [0, 1, 2, 3, 4, 5]
    assert G.seen_keys(10, 5, 3, parents=tree) == [0, 1, 2, 3, 4, 5, 6, 8]
    assert G.seen_keys(10, 5, 2, parents=tree) == [0, 1, 2, 3, 4, 5, 7]
    assert G.seen_keys(10, 5, 4, parents=tree) == [0, 1, 2, 3, 4, 9]
    # node 3 is at position 7: a window of 4 begins at 4 and holds its whole line
    assert G.seen_keys(10, 5, 3, 4, 1, tree) == [0, 4, 5, 6, 8]
    assert G.seen_keys(10, 5, 3, 2, 0, tree) == [6, 8]
    # a line that is none
    for bad in ([0, 0], [-1, 1], [-1, -2], [-1, 7]):
        assert G.seen_keys(10, 2, 1, parents=bad) == []
    assert G.seen_keys(1, 2, 1, parents=[-1, 0]) == []


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 0), (5, 3), (16, 16), (100, 0)])
def test_prompt_equals_the_library_with_a_mask(window, sinks):
    g = torch.Generator().manual_seed(window + sinks)
    new, keys, Hq, Hkv, d = [7, 1, 12], [20, 9, 12], 4, 2, 8
    q = torch.randn(sum(new), Hq, d, generator=g, dtype=torch.float64)
    k, v = (torch.randn(sum(keys), Hkv, d, generator=g, dtype=torch.float64) for _ in range(2))
    got = G.window_prompt(q, k, v, new, keys, 0.3, window, sinks)
    q0 = k0 = 0
    for n, nk in zip(new, keys):
        i = torch.arange(n)[:, None] + nk - n
        j = torch.arange(nk)
        mask = j <= i
        if window:
            mask = mask & ((i - j < window) | (j < sinks))
        ref = torch.nn.functional.scaled_dot_product_attention(
            q[q0:q0 + n].transpose(0, 1), k[k0:k0 + nk].transpose(0, 1).repeat_interleave(2, 0),
            v[k0:k0 + nk].transpose(0, 1).repeat_interleave(2, 0), attn_mask=mask, scale=0.3)
        np.testing.assert_allclose(got[q0:q0 + n], ref.transpose(0, 1).numpy(), atol=1e-12)
        q0, k0 = q0 + n, k0 + nk


def _cache(lens, Hkv, d, ps, seed):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    perm = torch.randperm(sum(need), generator=g)
    table = np.full((len(lens), max(need)), -7)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    k, v = (torch.randn(sum(need), Hkv, ps, d, generator=g, dtype=torch.float64).numpy() for _ in range(2))
    return k, v, table


def test_decode_without_a_mask_and_with_a_window_beyond_all_is_decode():
    lens = [5, 23, 40]
    k, v, table = _cache(lens, 2, 8, 16, 1)
    q = torch.randn(3, 3, 4, 8, generator=torch.Generator().manual_seed(2))
    ref = G.decode(q, k, v, None, None, table, lens, 0.4)
    for kw in ({}, dict(window=1000), dict(window=1000, sinks=3), dict(window=1, sinks=50),
               dict(parents=[[-1, 0, 1]] * 3)):
        np.testing.assert_allclose(
            G.decode_masked(q, k, v, None, None, table, lens, 0.4, **kw), ref, atol=1e-13)


def test_a_node_is_its_line_appended_as_a_chain():
    """Each node's row equals the last row of a chain: the tokens before the tree, then
    its line, stored one after the other; with a window too."""
    ps, n, tree = 16, 21, [-1, 0, 0, 1, 2, 2, -1, 6]
    Tq = len(tree)
    k, v, table = _cache([n], 1, 8, ps, 3)
    q = torch.randn(1, Tq, 2, 8, generator=torch.Generator().manual_seed(4))
    flat = [x[table[0]].transpose(0, 2, 1, 3).reshape(-1, 8) for x in (k, v)]
    for window, sinks in ((0, 0), (4, 0), (2, 3), (16, 1)):
        got = G.decode_masked(q, k, v, None, None, table, [n], 0.4, window, sinks, [tree])
        for t in range(Tq):
            line = [n - Tq + u for u in reversed(G.line_of(tree, t))]
            keys = list(range(n - Tq)) + line
            m = len(keys)
            row = G.window_prompt(q[0, t:t + 1], flat[0][keys][:, None], flat[1][keys][:, None], [1], [m],
                                  0.4, window, sinks)
            np.testing.assert_allclose(got[0, t], row[0], atol=1e-13)


def test_uniform_scores_give_means_of_the_seen_values():
    k, v, table = _cache([30], 1, 8, 16, 5)
    flat = v[table[0]].transpose(0, 2, 1, 3).reshape(-1, 8)
    got = G.decode_masked(np.zeros((1, 1, 1, 8)), k, v, None, None, table, [30], 1.0, 4, 2)
    np.testing.assert_allclose(got[0, 0, 0], flat[[0, 1, 26, 27, 28, 29]].mean(0), atol=1e-13)
