"""Ways of calling the paged-cache operators that their documentation allows:
in place, captured over changing tables, with tokens taken back."""
import numpy as np
import pytest
import torch

from oracle import paged as G
from tests.helpers import to64
from tests.test_gpu_paged import BF16, NR, Batch, _gen, attn_reference, check_append, run_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    assert torch.cuda.is_available()
    assert m.rf_get_device_status() == m.RF_OK
    return m


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("new", [[1, 1, 1], [5, 5, 5], [40, 0, 700]])
def test_append_with_queries_in_place(rf, kind, new):
    """q_out is q, a view of the rows that k and v are views of, too."""
    lens = [90, 33, 710]
    total = sum(new)
    bt = Batch(kind, lens, 2, 64, 32, seed=20)
    g = _gen(21)
    qkv = torch.randn(total, 10, 64, generator=g).to(BF16)
    nr = NR(rf, 64, 64, False, True, BF16, max_pos=800)
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
    cu = None if len(set(new)) == 1 else cu
    res = []
    for inplace in (False, True):
        cache = bt.device(rf)
        dev = qkv.cuda()
        q = dev[:, :6]
        out = q if inplace else torch.empty_like(q, memory_format=torch.contiguous_format)
        rf.rf_kv_append_paged(cache, dev[:, 6:8], dev[:, 8:], nr.dev,
                              None if cu is None else cu.cuda(), q, out)
        assert rf.rf_get_device_status() == rf.RF_OK
        res.append([t.clone() for t in (out, bt.k.t, bt.v.t, bt.ks, bt.vs) if t is not None])
        assert torch.equal(dev[:, 6:].cpu(), qkv[:, 6:])
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("lens,Tq,Hq", [([9000, 0, 17, 2500], 1, 8), ([40] * 300, 3, 6),
                                        ([5000, 300], 5, 8)])
def test_attn_in_place(rf, kind, lens, Tq, Hq):
    """O is Q: a tile's rows are written when all its parts have read them."""
    bt = Batch(kind, lens, 2, 64, 32, seed=22)
    cache = bt.device(rf)
    B = len(lens)
    q = torch.randn(B, Tq, Hq, 64, generator=_gen(23)).to(BF16)
    want, status = run_attn(rf, bt, q, 0.125, cache=cache)
    assert status == rf.RF_OK
    ws = torch.empty(rf.rf_attn_decode_paged_workspace_size(B, Hq, 2, Tq, 64), dtype=torch.uint8,
                     device="cuda")
    for _ in range(5):
        x = q.cuda()
        rf.rf_attn_decode_paged(cache, x, x, 0.125, ws)
        assert torch.equal(x, want)


def test_prompt_appends_in_a_graph_follow_their_tables(rf):
    """Lengths, tokens a sequence and the block table change between replays."""
    for kind in ("e4m3", "bf16"):
        nr = NR(rf, 128, 128, False, True, BF16, max_pos=400)
        total = 150
        rounds = [([200, 90, 0, 61], [99, 50, 0, 1]), ([30, 399, 120, 0], [20, 10, 120, 0]),
                  ([150, 0, 0, 0], [150, 0, 0, 0])]
        static = dict(k=torch.zeros(total, 2, 128, dtype=BF16, device="cuda"),
                      v=torch.zeros(total, 2, 128, dtype=BF16, device="cuda"),
                      q=torch.zeros(total, 3, 128, dtype=BF16, device="cuda"),
                      cu=torch.zeros(5, dtype=torch.int32, device="cuda"),
                      lens=torch.zeros(4, dtype=torch.int32, device="cuda"),
                      table=torch.zeros(4, 13, dtype=torch.int32, device="cuda"))
        out = torch.empty_like(static["q"])
        bts = [Batch(kind, lens, 2, 128, 32, seed=30 + i, max_pages=13)
               for i, (lens, _) in enumerate(rounds)]
        n = max(bt.num_pages for bt in bts)
        e = kind == "e4m3"
        pages = [torch.zeros(n, 2, 32, 128, dtype=torch.uint8 if e else BF16, device="cuda")
                 for _ in range(2)]
        scales = [torch.ones(n, 2, device="cuda") if e else None for _ in range(2)]
        cache = rf.rf_paged_kv(pages[0], pages[1], static["table"], static["lens"], *scales)

        def call():
            rf.rf_kv_append_paged(cache, static["k"], static["v"], nr.dev, static["cu"], static["q"],
                                  out)

        call()                                        # all sequences padded: nothing is written
        assert rf.rf_get_device_status() == rf.RF_ERR_DEVICE_INPUT     # cu_seqlens end below total
        assert not pages[0].any() and not pages[1].any()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for i, (lens, new) in enumerate(rounds):
            bt = bts[i]
            g = _gen(40 + i)
            x = {w: torch.randn(static[w].shape, generator=g).to(BF16) for w in "kvq"}
            for w in "kvq":
                static[w].copy_(x[w])
            static["cu"].copy_(torch.tensor([0] + new, dtype=torch.int32).cumsum(0))
            static["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            static["table"].copy_(bt.table)
            m = bt.num_pages
            for t in range(2):
                pages[t].zero_()
                pages[t][:m].copy_(torch.from_numpy(bt.pages[t]) if e else bt.pages[t])
                if e:
                    scales[t][:m].copy_(torch.from_numpy(bt.scale[t]))
            graph.replay()
            torch.cuda.synchronize()
            assert rf.rf_get_device_status() == rf.RF_OK
            # an eager call on a cache of its own gives the same bits and is the oracle's
            own = bt.device(rf)
            o2 = torch.empty_like(out)
            check_append(rf, bt, own, new, x["k"], x["v"], nr,
                         torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32), x["q"],
                         o2, f"round {i}")
            assert torch.equal(pages[0][:m], bt.k.t) and torch.equal(pages[1][:m], bt.v.t)
            if e:
                assert torch.equal(scales[0][:m], bt.ks) and torch.equal(scales[1][:m], bt.vs)
            rows = torch.cat([torch.full((c,), float(L > 0)) for L, c in zip(lens, new)]).bool()
            assert torch.equal(out.cpu()[rows], o2.cpu()[rows])


def test_tokens_taken_back_leave_their_scale(rf):
    """Loud draft tokens raise a page's scale; overwritten by quiet ones behind tokens
    that the page holds, the scale stays, and the values keep its coarser steps.  From
    slot 0 on the scale is the new tokens' own."""
    bt = Batch("e4m3", [16], 1, 64, 16, seed=50, loud=0.0)
    cache = bt.device(rf)
    g = _gen(51)
    quiet = torch.randn(2, 16, 1, 64, generator=g).to(BF16)
    loud = (64 * torch.randn(2, 8, 1, 64, generator=g)).to(BF16)

    def append(n, x):
        bt.dlens.fill_(n)
        rf.rf_kv_append_paged(cache, x[0].cuda(), x[1].cuda())

    append(16, quiet)
    first = bt.ks.clone(), bt.vs.clone()
    append(16, loud)                                  # slots 8 .. 15
    raised = bt.ks.clone(), bt.vs.clone()
    append(16, quiet[:, 8:])                          # taken back, and other tokens
    page = int(bt.table[0, 0])
    for w, (s, r, t, p) in enumerate(zip(first, raised, (bt.ks, bt.vs), (bt.k.t, bt.v.t))):
        assert r[page] > s[page] and t[page] == r[page]
        got = G.values(p.cpu().numpy(), t.cpu().numpy())[page, 0]
        x = to64(quiet[w])[:, 0]
        assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -4 * 2.0 ** -6 * float(r[page])).all()
    append(16, quiet)                                 # from slot 0: as the first time
    assert bt.ks[page] == first[0][page] and bt.vs[page] == first[1][page]
    assert rf.rf_get_device_status() == rf.RF_OK
