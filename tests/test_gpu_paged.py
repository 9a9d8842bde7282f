"""Paged-cache operators on the GPU against the fp64 oracle.

Tolerances, from the number formats (half a step of rounding is 2^-8 relative in
bf16, 2^-11 in fp16, 2^-24 in fp32, 2^-4 in E4M3):
* norm and rotation: one rounding to the output's type, plus fp32 arithmetic
  (a sum of d squares by fours and a tree, a reciprocal root, four products and
  an addition: under 32 steps of 2^-24) on terms no larger than twice the row's
  largest element;
* stored E4M3 codes: the code of a value within that arithmetic error of the
  exact one (values themselves, which have no arithmetic, exactly);
* attention: one rounding to bf16 of a sum of weights times values in which
  every weight carries the rounding of P (2^-11 in f16, 2^-16 as two bf16 parts),
  the error of its score (an fp32 sum of d products, and a few products and the
  exponential) and that of the running sums.  attn_reference adds these up.
"""
import numpy as np
import pytest
import torch

from oracle import paged as G
from oracle.fp8_quant_gemm import e4m3_decode, e4m3_encode
from tests.helpers import Guarded, to64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    assert torch.cuda.is_available()
    assert m.rf_get_device_status() == m.RF_OK
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _tables(max_pos, rot):
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)[None, :]
    return a.cos().float(), a.sin().float()


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def assert_rows(got, ref, dtype, what):
    got, ref = to64(got), np.asarray(ref)
    big = np.abs(ref).max(-1, keepdims=True)
    tol = _half(dtype) * np.abs(ref) + 32 * 2.0 ** -24 * 2 * big + 1e-37
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(got - ref).max()}"


class NR:
    """Norm and rotation on both sides."""

    def __init__(self, rf, d, rot, inter, norm, dtype, max_pos=600, seed=0):
        self.kw = {}
        cos = sin = wq = wk = None
        if rot:
            cos, sin = _tables(max_pos, rot)
        if norm:
            wq, wk = ((1 + 0.3 * torch.randn(d, generator=_gen(seed + i))).to(dtype) for i in (1, 2))
        c = [None if t is None else t.cuda() for t in (cos, sin, wq, wk)]
        self.dev = rf.rf_norm_rope(c[0], c[1], inter, c[2], c[3], 1e-5)
        self.cos, self.sin, self.inter, self.w = cos, sin, inter, {"q": wq, "k": wk}

    def ref(self, x, pos, which):
        return G.norm_rope(x, pos, self.cos, self.sin, self.inter, self.w[which], 1e-5)


# ------------------------------------------------------------------ norm and rotation


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot,inter,norm", [(128, 128, False, True), (128, 64, True, False),
                                              (128, 16, False, False), (64, 64, True, True),
                                              (64, 32, False, True), (64, 0, False, True),
                                              (128, 0, False, False), (64, 48, True, True),
                                              (128, 96, False, True)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (3, 5, 2), (67, 9, 3)])
def test_qk_norm_rope(rf, dtype, d, rot, inter, norm, T, Hq, Hkv):
    nr = NR(rf, d, rot, inter, norm, dtype)
    g = _gen(T + d + rot)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(dtype)
    pos = torch.randint(0, 600, (T,), generator=g, dtype=torch.int32)
    pos[0] = 599
    dev = qkv.cuda()
    qo, ko = Guarded((T, Hq, d), dtype), Guarded((T, Hkv, d), dtype)
    rf.rf_qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], qo.t, ko.t, nr.dev, pos.cuda())
    assert rf.rf_get_device_status() == rf.RF_OK
    assert_rows(qo.t, nr.ref(qkv[:, :Hq], pos, "q"), dtype, "q")
    assert_rows(ko.t, nr.ref(qkv[:, Hq:Hq + Hkv], pos, "k"), dtype, "k")
    qo.check("q")
    ko.check("k")
    # in place on the fused projection's rows: the same bits, the values untouched
    rf.rf_qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, :Hq], dev[:, Hq:Hq + Hkv], nr.dev,
                       pos.cuda())
    assert torch.equal(dev[:, :Hq], qo.t) and torch.equal(dev[:, Hq:Hq + Hkv], ko.t)
    assert torch.equal(dev[:, Hq + Hkv:].cpu(), qkv[:, Hq + Hkv:])


@pytest.mark.parametrize("T", [1, 700, 5000])
def test_qk_norm_rope_many_tokens_one_side_only(rf, T):
    nr = NR(rf, 128, 128, False, True, BF16)
    x = torch.randn(T, 7, 128, generator=_gen(T)).to(BF16)
    pos = torch.arange(T, dtype=torch.int32) % 600
    a, b = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), None, a, None, nr.dev, pos.cuda())
    rf.rf_qk_norm_rope(None, x.cuda(), None, b, nr.dev, pos.cuda())
    assert_rows(a, nr.ref(x, pos, "q"), BF16, "q alone")
    assert_rows(b, nr.ref(x, pos, "k"), BF16, "k alone")


def test_qk_norm_of_the_queries_only(rf):
    nr = NR(rf, 64, 64, False, True, BF16)
    only_q = rf.rf_norm_rope(nr.dev.cos, nr.dev.sin, False, nr.dev.q_weight, None, 1e-5)
    x = torch.randn(33, 3, 64, generator=_gen(5)).to(BF16)
    pos = torch.arange(33, dtype=torch.int32)
    a, b = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), x.cuda(), a, b, only_q, pos.cuda())
    assert_rows(a, nr.ref(x, pos, "q"), BF16, "q")
    assert_rows(b, G.norm_rope(x, pos, nr.cos, nr.sin), BF16, "k, no norm")


def test_qk_norm_rope_magnitudes_and_nonfinite_rows(rf):
    """Large and tiny rows, a zero row; an infinity or NaN stays in its row."""
    nr = NR(rf, 128, 128, False, True, BF16)
    x = torch.randn(8, 2, 128, generator=_gen(6))
    x[0] *= 1e15
    x[1] *= 1e-18
    x[2] = 0
    x[3, 0, 5] = float("inf")
    x[4, 1, 7] = float("nan")
    x = x.to(BF16)
    pos = torch.arange(8, dtype=torch.int32)
    o = torch.empty_like(x, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), None, o, None, nr.dev, pos.cuda())
    ref, got = nr.ref(x, pos, "q"), to64(o)
    keep = np.ones((8, 2), bool)
    keep[3, 0] = keep[4, 1] = False
    assert_rows(got[keep], ref[keep], BF16, "finite rows")
    assert np.isnan(got[4, 1]).all() and np.isnan(got[3, 0]).any()


def test_qk_positions_outside_the_tables(rf):
    nr = NR(rf, 64, 64, False, False, BF16)
    x = torch.randn(6, 2, 64, generator=_gen(7)).to(BF16)
    pos = torch.tensor([0, -1, 5, 600, 2**31 - 1, 599], dtype=torch.int32)
    o = torch.full_like(x, 7.0, device="cuda")
    rf.rf_qk_norm_rope(x.cuda(), None, o, None, nr.dev, pos.cuda())
    assert rf.rf_get_device_status() == rf.RF_ERR_DEVICE_INPUT
    assert rf.rf_get_device_status() == rf.RF_OK
    assert (o[[1, 3, 4]] == 7.0).all()
    ok = [0, 2, 5]
    assert_rows(o[ok], nr.ref(x[ok], pos[ok], "q"), BF16, "tokens inside")


# ------------------------------------------------------------------ append


class Batch:
    """A cache on both sides.  Pages that hold tokens behave; everything else is
    garbage (NaN codes and scales, random table entries)."""

    def __init__(self, kind, lens, Hkv, d, ps, seed=0, max_pages=None, loud=1.0):
        g = _gen(seed)
        need = [max(0, -(-n // ps)) for n in lens]
        self.B, self.ps, self.Hkv, self.d, self.kind, self.lens = len(lens), ps, Hkv, d, kind, lens
        self.num_pages = sum(need) + 2
        mp = max_pages or max(need + [1])
        perm = torch.randperm(self.num_pages, generator=g)
        self.table = torch.randint(-9, 10**6, (self.B, mp), generator=g, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (self.num_pages, Hkv, ps, d)
        x = torch.randn(2, *shape, generator=g) * torch.exp(
            loud * torch.randn(2, self.num_pages, Hkv, 1, 1, generator=g))
        if kind == "e4m3":
            self.scale = np.array([[[G.pow2_scale(float(a)) for a in row] for row in t]
                                   for t in x.abs().amax((3, 4)).numpy()], np.float32)
            self.pages = e4m3_encode(x.numpy() / self.scale[..., None, None])
        else:
            self.scale = None
            self.pages = x.to(BF16)

    def garbage(self):
        """Fills what no sequence holds."""
        held = np.zeros((self.num_pages, self.ps), bool)
        for b, n in enumerate(self.lens):
            for i in range(max(0, -(-n // self.ps))):
                held[int(self.table[b, i]), :min(self.ps, n - i * self.ps)] = True
        for t in range(2):
            if self.kind == "e4m3":
                self.pages[t].transpose(0, 2, 1, 3)[~held] = 0x7F
                self.scale[t][~held.any(1)] = np.nan
            else:
                self.pages[t].permute(0, 2, 1, 3)[torch.from_numpy(~held)] = float("nan")
        return self

    def device(self, rf, lens=None):
        e = self.kind == "e4m3"
        p = [(torch.from_numpy(t) if e else t).contiguous() for t in self.pages]
        self.k, self.v = (Guarded(tuple(t.shape), t.dtype) for t in p)
        self.k.t.copy_(p[0])
        self.v.t.copy_(p[1])
        s = [torch.from_numpy(t.copy()).cuda() if e else None for t in (self.scale if e else (0, 0))]
        self.ks, self.vs = s
        self.dlens = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32).cuda()
        return rf.rf_paged_kv(self.k.t, self.v.t, self.table.cuda(), self.dlens, *s)

    def host(self, which):
        """(pages, scale) as the oracle takes them."""
        return (self.pages[which], self.scale[which]) if self.kind == "e4m3" else \
            (to64(self.pages[which]), None)


def check_append(rf, bt, cache, new, k, v, nr, cu, q=None, q_out=None, what=""):
    """Runs the append and compares every byte of the cache with the oracle's."""
    k0, ks0 = bt.host(0)
    v0, vs0 = bt.host(1)
    rf.rf_kv_append_paged(cache, k.cuda(), v.cuda(), nr.dev if nr else None,
                          None if cu is None else cu.cuda(), None if q is None else q.cuda(), q_out)
    assert rf.rf_get_device_status() == rf.RF_OK, what
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(bt.lens, new)] + [np.zeros(0, int)])
    pos = np.maximum(pos, 0).astype(int)                  # padded rows: not looked at
    kr = nr.ref(k, pos, "k") if nr else to64(k)
    k1, v1, ks1, vs1 = G.append(k0, v0, ks0, vs0, bt.table.numpy(), bt.lens, new, kr, v)
    bt.k.check(what)
    bt.v.check(what)
    if bt.kind == "e4m3":
        np.testing.assert_array_equal(bt.ks.cpu().numpy(), ks1.astype(np.float32), err_msg=what)
        np.testing.assert_array_equal(bt.vs.cpu().numpy(), vs1.astype(np.float32), err_msg=what)
        np.testing.assert_array_equal(bt.v.t.cpu().numpy(), v1, err_msg=what)
        got = bt.k.t.cpu().numpy()
        off = got != k1
        if off.any():               # only where the exact value is that near to a border
            assert nr is not None, what
            scale = np.broadcast_to(ks1[:, :, None, None], got.shape)
            # rows' largest element is at most 448 scales of its page
            err = 64 * 2.0 ** -24 * 448
            x = exact_keys(bt, new, kr, k0.shape) / scale
            lo, hi = e4m3_decode(e4m3_encode(x - err)), e4m3_decode(e4m3_encode(x + err))
            val = e4m3_decode(got)
            assert ((val >= lo) & (val <= hi))[off].all(), what
            assert off.mean() < 1e-3, what
    else:
        np.testing.assert_array_equal(
            bt.v.t.cpu().view(torch.int16).numpy(),
            torch.from_numpy(v1).to(BF16).view(torch.int16).numpy(), err_msg=what)
        x = exact_keys(bt, new, kr, k0.shape)
        fresh = ~np.isnan(x)
        got = to64(bt.k.t)
        np.testing.assert_array_equal(got[~fresh], k0[~fresh], err_msg=what)
        big = np.abs(kr).max() if kr.size else 0.0
        assert (np.abs(got - x)[fresh] <= (2.0 ** -8 * np.abs(x) + 64 * 2.0 ** -24 * big)[fresh]).all()


def exact_keys(bt, new, kr, shape):
    """The new keys' exact values where they are stored; NaN elsewhere."""
    x = np.full(shape, np.nan)
    t = 0
    for b, m in enumerate(new):
        for i in range(m):
            p = bt.lens[b] - m + i
            if bt.lens[b]:
                x[int(bt.table[b, p // bt.ps]), :, p % bt.ps] = kr[t]
            t += 1
    return x


APPENDS = [
    # kind, page size, d, Hkv, lens after, new, cu, (rot, interleaved, norm)
    ("e4m3", 64, 128, 2, [1, 64, 65, 128, 300, 0, 17], [1] * 7, False, (128, False, True)),
    ("e4m3", 16, 64, 3, [1, 16, 17, 32, 33, 0], [1] * 6, False, (64, True, False)),
    ("e4m3", 128, 128, 1, [128, 129, 127], [1] * 3, False, None),
    ("bf16", 32, 128, 2, [1, 32, 33, 0, 100], [1] * 5, False, (64, False, True)),
    ("bf16", 16, 64, 5, [16, 17], [1] * 2, False, (32, False, False)),
    ("e4m3", 64, 128, 2, [150, 64, 3, 0, 200, 77], [150, 0, 3, 0, 63, 5], True, (128, False, True)),
    ("e4m3", 16, 128, 2, [100, 1, 16, 40], [37, 1, 16, 30], True, (16, True, True)),
    ("e4m3", 32, 64, 4, [70, 64, 33], [64, 1, 33], True, (64, False, False)),
    ("e4m3", 128, 64, 2, [300, 129, 5], [200, 2, 5], True, None),
    ("e4m3", 128, 128, 1, [500, 256], [500, 129], True, (128, True, True)),
    ("bf16", 64, 128, 3, [150, 1, 200], [130, 1, 64], True, (128, False, True)),
    ("bf16", 128, 64, 2, [300, 10], [299, 10], True, (64, True, True)),
    ("bf16", 16, 128, 1, [45, 18, 0], [20, 18, 2], True, (96, False, False)),
    ("e4m3", 64, 128, 2, [90, 64, 7, 0], [5] * 4, False, (128, False, True)),
    ("bf16", 32, 64, 2, [33, 66], [33] * 2, False, (64, False, True)),
    ("e4m3", 16, 128, 3, [8, 19, 40, 0, 16, 17, 24], [8] * 7, False, (128, False, True)),
    ("e4m3", 64, 64, 5, [3, 66, 65, 0, 64, 67], [3] * 6, False, (32, True, False)),
    ("e4m3", 32, 128, 2, [9, 40, 33, 32], [9] * 4, False, (128, False, True)),
    ("e4m3", 128, 64, 2, [2, 129], [2] * 2, False, (64, False, True)),
]


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(rf, case):
    kind, ps, d, Hkv, lens, new, use_cu, rope = APPENDS[case]
    total = sum(new)
    bt = Batch(kind, lens, Hkv, d, ps, seed=case)
    cache = bt.device(rf)
    g = _gen(100 + case)
    Hq = 3 * Hkv
    # louder than what the pages hold, so that some of them are rescaled
    qkv = torch.randn(total, Hq + 2 * Hkv, d, generator=g) * torch.exp(
        1.5 * torch.randn(total, Hq + 2 * Hkv, 1, generator=g))
    qkv = qkv.to(BF16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    nr = NR(rf, d, rope[0], rope[1], rope[2], BF16, seed=case) if rope else None
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32) if use_cu else None
    q_out = Guarded((total, Hq, d), BF16, fill=7.0)
    check_append(rf, bt, cache, new, k, v, nr, cu, q, q_out.t, f"append {case}")
    q_out.check("q_out")
    t = 0
    for n, m in zip(lens, new):
        rows = slice(t, t + m)
        t += m
        if n == 0:
            assert (q_out.t[rows] == 7.0).all(), "rows of a padded sequence"
        elif m:
            pos = np.arange(n - m, n)
            ref = nr.ref(q[rows], pos, "q") if nr else to64(q[rows])
            assert_rows(q_out.t[rows], ref, BF16, "q")


def test_append_reads_strided_views_and_equals_dense(rf):
    bt = Batch("e4m3", [40, 70], 2, 128, 32, seed=50)
    g = _gen(51)
    qkv = torch.randn(2, 11, 128, generator=g).to(BF16).cuda()
    nr = NR(rf, 128, 128, False, True, BF16)
    res = []
    for dense in (False, True):
        cache = bt.device(rf)
        k, v = qkv[:, 3:5], qkv[:, 9:11]
        rf.rf_kv_append_paged(cache, k.contiguous() if dense else k, v.contiguous() if dense else v,
                              nr.dev)
        res.append([t.clone() for t in (bt.k.t, bt.v.t, bt.ks, bt.vs)])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_append_nonfinite_and_zero_values(rf):
    bt = Batch("e4m3", [1, 5, 20], 1, 64, 16, seed=52)
    cache = bt.device(rf)
    k = torch.randn(3, 1, 64, generator=_gen(53))
    v = torch.randn(3, 1, 64, generator=_gen(54))
    v[0, 0, 3], v[0, 0, 4], v[0, 0, 5] = float("inf"), -float("inf"), float("nan")
    v[1] = 0
    k[2] = float("nan")
    v[2] = torch.finfo(BF16).max
    check_append(rf, bt, cache, [1, 1, 1], k.to(BF16), v.to(BF16), None, None, what="non-finite")


def test_append_repeats_and_token_by_token(rf):
    """The same call again changes nothing; growing a cache a token at a time
    keeps it what the oracle's growth makes it."""
    B, Hkv, d, ps, n = 3, 2, 128, 16, 40
    bt = Batch("e4m3", [n] * B, Hkv, d, ps, seed=55)
    bt.lens = [0] * B
    cache = bt.device(rf)
    g = _gen(56)
    xs = [(torch.randn(2, B, Hkv, d, generator=g) * torch.exp(torch.randn(B, 1, 1, generator=g))).to(BF16)
          for _ in range(n)]
    for t, x in enumerate(xs):
        bt.lens = [t + 1] * B
        bt.dlens.add_(1)
        check_append(rf, bt, cache, [1] * B, x[0], x[1], None, None, what=f"token {t}")
        bt.pages = np.stack([bt.k.t.cpu().numpy(), bt.v.t.cpu().numpy()])
        bt.scale = np.stack([bt.ks.cpu().numpy(), bt.vs.cpu().numpy()])
    before = [t.clone() for t in (bt.k.t, bt.v.t, bt.ks, bt.vs)]
    rf.rf_kv_append_paged(cache, xs[-1][0].cuda(), xs[-1][1].cuda())
    assert all(torch.equal(a, b) for a, b in zip(before, (bt.k.t, bt.v.t, bt.ks, bt.vs)))


@pytest.mark.parametrize("use_cu", [False, True])
def test_append_inconsistent_sequences_are_skipped(rf, use_cu):
    """Lengths and pages that do not fit: reported, skipped, the others done."""
    lens = [40, 3, 20, 33, 30]
    bt = Batch("e4m3", lens, 2, 64, 16, seed=57, max_pages=3)
    new = [2] * 5
    told = [40, 1, 10**6, 33, -5]            # 1: shorter than its new tokens
    bt.table[3, 2] = bt.num_pages            # sequence 3's last page: token 33 (slot 0)
    cache = bt.device(rf, told)
    g = _gen(58)
    k, v = (torch.randn(10, 2, 64, generator=g).to(BF16) for _ in range(2))
    q = torch.randn(10, 4, 64, generator=g).to(BF16)
    q_out = torch.full((10, 4, 64), 7.0, dtype=BF16, device="cuda")
    cu = torch.arange(0, 11, 2, dtype=torch.int32).cuda() if use_cu else None
    rf.rf_kv_append_paged(cache, k.cuda(), v.cuda(), None, cu, q.cuda(), q_out)
    assert rf.rf_get_device_status() == rf.RF_ERR_DEVICE_INPUT
    # oracle: sequence 0 whole, of sequence 3 the token at position 31 only
    k0, v0, ks0, vs0 = bt.pages[0], bt.pages[1], bt.scale[0], bt.scale[1]
    ref = G.append(k0, v0, ks0, vs0, bt.table.numpy(), [40], [2], k[:2], v[:2])
    ref = G.append(*ref, bt.table.numpy()[3:4], [32], [1], k[6:7], v[6:7])
    for got, want in zip((bt.k.t, bt.v.t, bt.ks, bt.vs), ref):
        np.testing.assert_array_equal(got.cpu().numpy(), want.astype(got.cpu().numpy().dtype))
    skipped = [2, 3, 4, 5, 8, 9]
    assert (q_out[skipped] == 7.0).all()
    assert torch.equal(q_out[[0, 1, 6, 7]].cpu(), q[[0, 1, 6, 7]])


@pytest.mark.parametrize("between,tokens", [(1, 100), (41, 2000)])
def test_append_of_tokens_that_several_sequences_claim(rf, between, tokens):
    """cu_seqlens that fall back to 0: the first and the last sequence claim the
    same tokens, and (in one warp, and in two) some of the same items.  Reported;
    a page is left alone or gets what one of them appends, never a mixture."""
    B = between + 2
    lens = [tokens] + [0] * between + [tokens]
    bt = Batch("e4m3", lens, 2, 64, 16, seed=59)
    cache = bt.device(rf, lens)
    cu = [0] + [tokens] * between + [0, tokens]
    claims = [set(range(c // 16 + 2 * b, c // 16 + 2 * b + -(-tokens // 16)))
              for b, c in ((0, 0), (B - 1, 0))]
    assert claims[0] & claims[1]
    g = _gen(60)
    k, v = (torch.randn(tokens, 2, 64, generator=g).to(BF16) for _ in range(2))
    rf.rf_kv_append_paged(cache, k.cuda(), v.cuda(), None,
                          torch.tensor(cu, dtype=torch.int32).cuda())
    assert rf.rf_get_device_status() == rf.RF_ERR_DEVICE_INPUT
    before = (bt.pages[0], bt.pages[1], bt.scale[0], bt.scale[1])
    after = before
    for b in (0, B - 1):
        after = G.append(*after, bt.table.numpy()[b:b + 1], [tokens], [tokens], k, v)
    got = [t.cpu().numpy() for t in (bt.k.t, bt.v.t, bt.ks, bt.vs)]
    n = bt.num_pages
    same = [[(x[i] == y[i].astype(x.dtype)).all() for i in range(n)] for ref in (before, after)
            for x, y in zip(got, ref)]
    left, done = np.array(same[:4]).all(0), np.array(same[4:]).all(0)
    assert (left | done).all()
    own = [bt.table.numpy()[b, :-(-tokens // 16)] for b in (0, B - 1)]
    first = sorted(claims[0] - claims[1])            # items of the first sequence alone
    assert done[own[0][first]].all()
    last = sorted(x - min(claims[1]) for x in claims[1] - claims[0])
    assert done[own[1][last]].all()
    bt.k.check("k")
    bt.v.check("v")


# ------------------------------------------------------------------ attention


def attn_reference(q, bt, scale):
    """(o, tolerance) in fp64, vectorised over the rows of a kv head; the sum of
    the kernel's error bounds as the file's head lists them."""
    q = to64(q)
    B, Tq, Hq, d = q.shape
    K, V = (G.values(*bt.host(i)) for i in (0, 1))
    e4m3 = bt.kind == "e4m3"
    G_ = Hq // bt.Hkv
    o, tol = np.zeros_like(q), np.zeros_like(q)
    u = 2.0 ** -23                                   # one fp32 operation, not assumed to round
    for b, n in enumerate(bt.lens):
        if n <= 0:
            continue
        pages = bt.table[b, :-(-n // bt.ps)].numpy()
        for h in range(bt.Hkv):
            kb, vb = (x[pages, h].reshape(-1, d)[:n] for x in (K, V))
            vs = np.repeat(bt.scale[1][pages, h], bt.ps)[:n] if e4m3 else np.ones(n)
            for t in range(Tq):
                m = max(0, n - Tq + t + 1)
                if m == 0:
                    continue
                rows = slice(h * G_, (h + 1) * G_)
                qr = q[b, t, rows]
                s = scale * qr @ kb[:m].T
                size = scale * np.abs(qr) @ np.abs(kb[:m]).T
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                va = np.abs(vb[:m])
                # natural-log error of a weight: score, products, exponential
                e = (d + 8) * u * size.max(1) + 4 * u * np.abs(s).max(1) + 8 * u
                per = 2 * e + (2.0 ** -11 if e4m3 else 2.0 ** -16) + (m / 8 + 64) * u
                o[b, t, rows] = p @ vb[:m]
                tol[b, t, rows] = per[:, None] * (p @ va)
                if e4m3:                             # weights that fall into f16's subnormals
                    w = p * vs[:m]
                    top = w.max(1, keepdims=True)
                    small = w < 2.0 ** -14 * top
                    tol[b, t, rows] += 2.0 ** -25 * top * (small @ (va / vs[:m, None]))
    return o, tol + 2.0 ** -8 * (np.abs(o) + tol) + 1e-37


def run_attn(rf, bt, q, scale, ws=None, cache=None):
    cache = cache or bt.device(rf)
    B, Tq, Hq, d = q.shape
    o = Guarded((B, Tq, Hq, d), BF16)
    n = rf.rf_attn_decode_paged_workspace_size(B, Hq, bt.Hkv, Tq, d)
    ws = ws if ws is not None else Guarded((n,), torch.uint8, fill=0xFF)
    rf.rf_attn_decode_paged(cache, q.cuda(), o.t, scale, ws.t if isinstance(ws, Guarded) else ws)
    status = rf.rf_get_device_status()
    o.check("output")
    if isinstance(ws, Guarded):
        ws.check("workspace")
    return o.t, status


def check_attn(rf, bt, q, scale, what):
    got, status = run_attn(rf, bt, q, scale)
    assert status == rf.RF_OK, what
    ref, tol = attn_reference(q, bt, scale)
    got = to64(got)
    assert np.isfinite(got).all(), what
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside; worst "
                           f"{(np.abs(got - ref) / tol).max():.2f} of the tolerance")


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 64, 65, 127, 400]
ATTNS = [
    # kind, page size, d, Hkv, Hq, Tq, lens
    ("e4m3", 64, 128, 2, 8, 1, LENS), ("e4m3", 16, 128, 1, 5, 1, LENS),
    ("e4m3", 32, 64, 2, 16, 1, LENS), ("e4m3", 128, 64, 1, 9, 1, LENS),
    ("e4m3", 16, 64, 1, 16, 1, LENS), ("e4m3", 128, 128, 1, 33, 1, LENS),
    ("bf16", 64, 128, 2, 8, 1, LENS), ("bf16", 16, 128, 1, 7, 1, LENS),
    ("bf16", 32, 64, 3, 3, 1, LENS), ("bf16", 16, 64, 1, 17, 1, LENS),
    ("bf16", 128, 128, 1, 16, 1, LENS),
    ("e4m3", 64, 128, 2, 8, 2, LENS), ("e4m3", 16, 128, 1, 8, 4, LENS),
    ("e4m3", 32, 64, 1, 1, 7, LENS), ("e4m3", 64, 64, 1, 3, 40, LENS),
    ("bf16", 32, 128, 1, 2, 5, LENS), ("bf16", 16, 64, 2, 8, 3, LENS),
    ("bf16", 64, 128, 1, 1, 33, LENS),
    # long: tiles cut between warps and between CTAs
    ("e4m3", 64, 128, 2, 8, 1, [9000, 3, 20000]), ("e4m3", 16, 64, 1, 4, 1, [30001]),
    ("bf16", 32, 128, 1, 8, 1, [25000]), ("bf16", 128, 64, 2, 2, 2, [11111, 0, 7777]),
    ("e4m3", 16, 128, 1, 12, 3, [15000, 100]),
    # many short ones: tiles that begin and end inside a warp's range
    ("e4m3", 16, 128, 4, 4, 1, [1 + i % 40 for i in range(700)]),
    ("bf16", 16, 64, 8, 8, 1, [(7 * i) % 70 for i in range(300)]),
]


@pytest.mark.parametrize("case", range(len(ATTNS)))
def test_attn_decode_paged(rf, case):
    kind, ps, d, Hkv, Hq, Tq, lens = ATTNS[case]
    bt = Batch(kind, lens, Hkv, d, ps, seed=200 + case).garbage()
    q = torch.randn(len(lens), Tq, Hq, d, generator=_gen(300 + case)).to(BF16)
    check_attn(rf, bt, q, d ** -0.5, f"attention {ATTNS[case][:6]}")


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_attn_equals_the_oracle_of_every_row(rf, kind):
    """The vectorised reference is the oracle's."""
    bt = Batch(kind, [5, 40, 0], 2, 64, 16, seed=240)
    q = torch.randn(3, 2, 4, 64, generator=_gen(241)).to(BF16)
    k, ks = bt.host(0)
    v, vs = bt.host(1)
    ref = G.decode(q, k, v, ks, vs, bt.table.numpy(), bt.lens, 0.125)
    np.testing.assert_allclose(attn_reference(q, bt, 0.125)[0], ref, atol=1e-12)
    check_attn(rf, bt, q, 0.125, kind)


@pytest.mark.parametrize("q_exp,k_exp,v_exp", [(60, -60, 0), (-60, 60, 0), (0, 0, 100), (0, 0, -100),
                                               (-130, 100, 0)])
def test_attn_scales_far_from_one(rf, q_exp, k_exp, v_exp):
    bt = Batch("e4m3", [100, 70], 2, 128, 16, seed=250)
    bt.scale[0] *= np.float32(2.0 ** k_exp)
    bt.scale[1] *= np.float32(2.0 ** v_exp)
    q = (torch.randn(2, 1, 8, 128, generator=_gen(251)) * 2.0 ** q_exp).to(BF16)
    check_attn(rf, bt, q, 128 ** -0.5, f"exponents {q_exp} {k_exp} {v_exp}")


def test_attn_pages_of_very_different_value_scales(rf):
    """A page of huge values that gets almost no weight beside one of small
    values that gets almost all: neither may drown the other."""
    bt = Batch("e4m3", [64, 200], 1, 64, 16, seed=252)
    for b in range(2):
        for i in range(-(-bt.lens[b] // 16)):
            bt.scale[1][int(bt.table[b, i])] = np.float32(2.0 ** [0, 20, -30, 40, 3.5][i % 5])
    q = 6 * torch.randn(2, 1, 4, 64, generator=_gen(253)).to(BF16)
    check_attn(rf, bt, q, 0.125, "value scales")


@pytest.mark.parametrize("q_exp", [0, -12, -60, -126])
def test_attn_pages_of_zeros(rf, q_exp):
    """Zero keys (the smallest scale), zero values, and queries so small that the
    product of all factors underflows; the last page is cut short."""
    for Tq in (1, 3):
        bt = Batch("e4m3", [5, 37, 64], 1, 64, 16, seed=256).garbage()
        for b, n in enumerate(bt.lens):
            page = int(bt.table[b, (n - 1) // 16])
            bt.pages[0][page, 0, :(n - 1) % 16 + 1] = 0
            bt.scale[0][page] = np.float32(2.0 ** -126)
        bt.pages[1][int(bt.table[1, 0])] = 0
        bt.scale[1][int(bt.table[1, 0])] = np.float32(2.0 ** -126)
        q = (torch.randn(3, Tq, 4, 64, generator=_gen(257)) * 2.0 ** q_exp).to(BF16)
        check_attn(rf, bt, q, 0.125, f"zeros, queries of 2^{q_exp}")


def test_attn_scales_that_are_no_powers_of_two(rf):
    bt = Batch("e4m3", [300], 2, 128, 64, seed=254)
    bt.scale *= np.float32(1.2345)
    q = torch.randn(1, 1, 16, 128, generator=_gen(255)).to(BF16)
    check_attn(rf, bt, q, 0.0884, "odd scales")


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("Tq,Hq", [(3, 2), (5, 16)])
def test_attn_a_draft_token_that_is_not_finite(rf, kind, Tq, Hq):
    """A non-finite key or value of a later token has no effect on the rows of
    earlier ones; the rows that read it are not finite."""
    bt = Batch(kind, [40, 33], 1, 64, 16, seed=260)
    clean = bt.pages.copy() if kind == "e4m3" else bt.pages.clone()
    q = torch.randn(2, Tq, Hq, 64, generator=_gen(261)).to(BF16)
    ref, tol = attn_reference(q, bt, 0.125)
    for which in (0, 1):
        bt.pages = clean.copy() if kind == "e4m3" else clean.clone()
        for b, n in enumerate(bt.lens):
            page, slot = int(bt.table[b, (n - 2) // 16]), (n - 2) % 16
            bt.pages[which][page, 0, slot] = 0x7F if kind == "e4m3" else float("inf")
        got, status = run_attn(rf, bt, q, 0.125)
        assert status == rf.RF_OK
        got = to64(got)
        assert (np.abs(got - ref) <= tol)[:, :Tq - 2].all(), "rows that do not read it"
        assert not np.isfinite(got[:, Tq - 2:]).all(-1).any(), "rows that read it"


def test_attn_a_query_that_is_not_finite_spoils_its_row_only(rf):
    for kind in ("e4m3", "bf16"):
        bt = Batch(kind, [50], 1, 128, 32, seed=262)
        q = torch.randn(1, 1, 8, 128, generator=_gen(263)).to(BF16)
        ref, tol = attn_reference(q, bt, 0.1)
        q[0, 0, 2, 5] = float("nan")
        q[0, 0, 6, 9] = float("inf")
        got = to64(run_attn(rf, bt, q, 0.1)[0])
        ok = [0, 1, 3, 4, 5, 7]
        assert (np.abs(got - ref) <= tol)[0, 0, ok].all() and np.isnan(got[0, 0, [2, 6]]).all()


def test_attn_inconsistent_lengths_and_pages(rf):
    """Reported, and taken as empty; other sequences keep their results."""
    lens = [100, 50, 70, 20]
    for kind in ("e4m3", "bf16"):
        bt = Batch(kind, lens, 2, 64, 16, seed=264)
        q = torch.randn(4, 1, 4, 64, generator=_gen(265)).to(BF16)
        cache = bt.device(rf, [100, -1, 10**9, 20])
        got, status = run_attn(rf, bt, q, 0.125, cache=cache)
        assert status == rf.RF_ERR_DEVICE_INPUT
        bt.lens = [100, 0, 0, 20]
        ref, tol = attn_reference(q, bt, 0.125)
        assert (np.abs(to64(got) - ref) <= tol).all()
        # a page outside the cache: its keys are absent
        bt.lens = [100, 50, 70, 20]
        good = bt.table.clone()
        bt.table[0, 3] = bt.num_pages
        bt.table[3, 0], bt.table[3, 1] = -1, 2**31 - 1       # all of sequence 3
        got, status = run_attn(rf, bt, q, 0.125)
        assert status == rf.RF_ERR_DEVICE_INPUT
        bt.table = good
        bt.table[0] = torch.cat([good[0, :3], good[0, 4:], good[0, 3:4]])
        bt.lens = [84, 50, 70, 0]                            # 100 keys less a page of 16
        ref, tol = attn_reference(q, bt, 0.125)
        assert (np.abs(to64(got) - ref) <= tol).all()


def test_attn_shared_pages_and_repeated_table_rows(rf):
    bt = Batch("e4m3", [90, 90, 90], 2, 64, 16, seed=266)
    bt.table[1] = bt.table[0]
    bt.table[2, 3] = bt.table[2, 0]                          # one page twice in a sequence
    q = torch.randn(3, 1, 4, 64, generator=_gen(267)).to(BF16)
    q[1] = q[0]
    check_attn(rf, bt, q, 0.125, "shared pages")


def test_attn_offsets_beyond_32_bits(rf):
    """A pool of 4.5 GB a tensor; the sequence lives in its last pages."""
    num_pages, ps, d = 140000, 128, 128
    pages = [torch.zeros(num_pages, 2, ps, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(num_pages, 2, device="cuda") for _ in range(2)]
    bt = Batch("e4m3", [700], 2, d, ps, seed=268)
    n = bt.num_pages
    base = num_pages - n
    for t in range(2):
        pages[t][base:] = torch.from_numpy(bt.pages[t]).cuda()
        scales[t][base:] = torch.from_numpy(bt.scale[t]).cuda()
    table = (bt.table + base).cuda()
    lens = torch.tensor([700], dtype=torch.int32, device="cuda")
    cache = rf.rf_paged_kv(pages[0], pages[1], table, lens, *scales)
    q = torch.randn(1, 1, 8, d, generator=_gen(269)).to(BF16)
    got, status = run_attn(rf, bt, q, 0.0884, cache=cache)
    assert status == rf.RF_OK
    ref, tol = attn_reference(q, bt, 0.0884)
    assert (np.abs(to64(got) - ref) <= tol).all()
    k, v = (torch.randn(1, 2, d, generator=_gen(270 + i)).to(BF16) for i in range(2))
    rf.rf_kv_append_paged(cache, k.cuda(), v.cuda())
    assert rf.rf_get_device_status() == rf.RF_OK
    want = G.append(bt.pages[0], bt.pages[1], bt.scale[0], bt.scale[1], bt.table.numpy(), [700], [1],
                    k, v)
    np.testing.assert_array_equal(pages[0][base:].cpu().numpy(), want[0])
    np.testing.assert_array_equal(pages[1][base:].cpu().numpy(), want[1])
    assert not pages[0][:base].any() and not pages[1][:base].any()


# ------------------------------------------------------------------ together


def _step(rf, bt, cache, nr, qkv, q_out, o, ws, Hq, Hkv):
    rf.rf_kv_append_paged(cache, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], nr.dev, None, qkv[:, :Hq],
                          q_out)
    rf.rf_attn_decode_paged(cache, q_out, o, 128 ** -0.5, ws)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_decode_steps_in_a_graph_equal_eager_ones(rf, kind):
    """Append and attention as a decode loop runs them: captured once, replayed
    while the lengths grow (one sequence joins late, one is padding); the same
    bits as eager calls, on a stream of its own; and each step's output is the
    oracle's for the cache it left."""
    B, Hq, Hkv, ps, steps = 4, 8, 2, 16, 20
    nr = NR(rf, 128, 128, False, True, BF16)
    ws = torch.empty(rf.rf_attn_decode_paged_workspace_size(B, Hq, Hkv, 1, 128), dtype=torch.uint8,
                     device="cuda")
    results = []
    for mode in ("eager", "graph"):
        bt = Batch(kind, [60, 40, 50, 30], Hkv, 128, ps, seed=400)
        lens = torch.tensor([33, 1, 15, 0], dtype=torch.int32)
        cache = bt.device(rf, lens.tolist())
        qkv = torch.zeros(B, Hq + 2 * Hkv, 128, dtype=BF16, device="cuda")
        q_out = torch.zeros(B, Hq, 128, dtype=BF16, device="cuda")
        o = torch.zeros(B, Hq, 128, dtype=BF16, device="cuda")
        graph, outs = None, []
        stream = torch.cuda.Stream()
        if mode == "graph":
            keep = [t.clone() for t in (bt.k.t, bt.v.t)] + \
                [t.clone() for t in (bt.ks, bt.vs) if t is not None]
            _step(rf, bt, cache, nr, qkv, q_out, o, ws, Hq, Hkv)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                _step(rf, bt, cache, nr, qkv, q_out, o, ws, Hq, Hkv)
            for t, x in zip([t for t in (bt.k.t, bt.v.t, bt.ks, bt.vs) if t is not None], keep):
                t.copy_(x)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for i in range(steps):
                qkv.copy_(torch.randn(B, Hq + 2 * Hkv, 128, generator=_gen(500 + i)).to(BF16))
                if graph:
                    graph.replay()
                else:
                    _step(rf, bt, cache, nr, qkv, q_out, o, ws, Hq, Hkv)
                outs.append(o.clone())
                if mode == "eager":
                    stream.synchronize()
                    bt.lens = bt.dlens.tolist()
                    e = kind == "e4m3"
                    bt.pages = np.stack([t.cpu().numpy() for t in (bt.k.t, bt.v.t)]) if e else \
                        torch.stack([bt.k.t.cpu(), bt.v.t.cpu()])
                    bt.scale = np.stack([bt.ks.cpu().numpy(), bt.vs.cpu().numpy()]) if e else None
                    ref, tol = attn_reference(q_out.cpu()[:, None], bt, 128 ** -0.5)
                    assert (np.abs(to64(o)[:, None] - ref) <= tol).all(), f"step {i}"
                grow = [1, 1, 1, 1 if i >= 5 else 0]
                bt.dlens.add_(torch.tensor(grow, dtype=torch.int32).cuda())
        stream.synchronize()
        assert rf.rf_get_device_status() == rf.RF_OK
        results.append(outs)
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a, b), f"step {i}: graph and eager differ"


def test_prompt_then_steps_match_attention_over_the_whole(rf):
    """A prompt's norm and rotation, its prefill attention, its append, then decode
    steps over the bf16 cache: the last row of the prefill equals the decode's."""
    H, d, n = 2, 64, 77
    nr = NR(rf, d, d, False, True, BF16)
    g = _gen(600)
    q, k, v = (torch.randn(n, H, d, generator=g).to(BF16).cuda() for _ in range(3))
    pos = torch.arange(n, dtype=torch.int32).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    rf.rf_qk_norm_rope(q, k, qo, ko, nr.dev, pos)
    o = torch.empty_like(q)
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    rf.rf_attn_fwd_varlen(qo, ko, v, o, cu, cu, n, d ** -0.5, 1)
    bt = Batch("bf16", [n], H, d, 16, seed=601)
    cache = bt.device(rf)
    q2 = torch.empty_like(q)
    rf.rf_kv_append_paged(cache, k, v, nr.dev, cu, q, q2)
    assert torch.equal(q2, qo), "the append's queries are rf_qk_norm_rope's"
    od = torch.empty(1, 3, H, d, dtype=BF16, device="cuda")
    ws = torch.empty(rf.rf_attn_decode_paged_workspace_size(1, H, H, 3, d), dtype=torch.uint8,
                     device="cuda")
    rf.rf_attn_decode_paged(cache, qo[None, -3:].contiguous(), od, d ** -0.5, ws)
    assert rf.rf_get_device_status() == rf.RF_OK
    # both are within 2e-2 and 5e-3 (relative) of the exact result
    assert (o[-3:].float() - od[0].float()).abs().max() <= 2e-2
    err = (o[-3:].double() - od[0].double()).norm() / o[-3:].double().norm()
    assert err <= 1e-2


def test_attn_is_deterministic_and_ignores_the_workspace(rf):
    bt = Batch("e4m3", [5000, 100, 2500, 7], 2, 128, 64, seed=700)
    cache = bt.device(rf)
    q = torch.randn(4, 1, 8, 128, generator=_gen(701)).to(BF16).cuda()
    n = rf.rf_attn_decode_paged_workspace_size(4, 8, 2, 1, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(12):
        o = torch.empty_like(q)
        ws.random_(0, 256)
        rf.rf_attn_decode_paged(cache, q, o, 0.0884, ws)
        first = o if first is None else first
        assert torch.equal(o, first), f"call {i}"
    with pytest.raises(rf.RFError) as e:
        rf.rf_attn_decode_paged(cache, q, o, 0.0884, ws[:n - 16])
    assert e.value.status == rf.RF_ERR_WORKSPACE
    assert rf.rf_get_device_status() == rf.RF_OK


def test_attn_refuses_an_expanded_workspace(rf):
    bt = Batch("bf16", [5], 1, 64, 16, seed=3)
    cache = bt.device(rf)
    q = torch.zeros(1, 1, 64, dtype=BF16, device="cuda")
    n = rf.rf_attn_decode_paged_workspace_size(1, 1, 1, 1, 64)
    with pytest.raises(ValueError, match="workspace"):
        rf.rf_attn_decode_paged(cache, q, torch.empty_like(q), 1.0,
                                torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n))


def test_two_streams_with_workspaces_of_their_own(rf):
    """Two caches at once on two streams, outputs as when run one by one."""
    sets = []
    for i in range(2):
        bt = Batch("e4m3", [6000, 300], 2, 128, 32, seed=710 + i)
        q = torch.randn(2, 1, 8, 128, generator=_gen(712 + i)).to(BF16).cuda()
        ws = torch.empty(rf.rf_attn_decode_paged_workspace_size(2, 8, 2, 1, 128), dtype=torch.uint8,
                         device="cuda")
        sets.append((bt.device(rf), q, torch.empty_like(q), ws, torch.cuda.Stream(), bt))
    alone = []
    for cache, q, o, ws, _, _ in sets:
        rf.rf_attn_decode_paged(cache, q, o, 0.0884, ws)
        torch.cuda.synchronize()
        alone.append(o.clone())
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for cache, q, o, ws, s, _ in sets:
            rf.rf_attn_decode_paged(cache, q, o, 0.0884, ws, stream=s)
    torch.cuda.synchronize()
    for (_, _, o, _, _, _), a in zip(sets, alone):
        assert torch.equal(o, a)


def test_binding_checks(rf):
    bt = Batch("e4m3", [20], 2, 64, 16, seed=720)
    cache = bt.device(rf)
    x = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    o = torch.zeros(1, 4, 64, dtype=BF16, device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    bad = [lambda: rf.rf_kv_append_paged(cache, x.float(), x), lambda: rf.rf_kv_append_paged(cache, x, x[:, :1]),
           lambda: rf.rf_kv_append_paged(cache, x.cpu(), x),
           lambda: rf.rf_kv_append_paged(cache, x.transpose(1, 2), x),
           lambda: rf.rf_kv_append_paged(cache, x, x, None, None, o, None),
           lambda: rf.rf_kv_append_paged(cache, x, x, None, torch.zeros(3, dtype=torch.int32, device="cuda")),
           lambda: rf.rf_kv_append_paged(cache, x, x, rf.rf_norm_rope(k_weight=torch.ones(64, device="cuda"))),
           lambda: rf.rf_attn_decode_paged(cache, o.float(), o, 0.1, ws),
           lambda: rf.rf_attn_decode_paged(cache, o, o[:, :2], 0.1, ws),
           lambda: rf.rf_attn_decode_paged(cache, o[..., :32], o, 0.1, ws),
           lambda: rf.rf_qk_norm_rope(x, None, x, None, rf.rf_norm_rope(
               torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda"))),
           lambda: rf.rf_qk_norm_rope(None, None, None, None, None),
           lambda: rf.rf_paged_kv(bt.k.t, bt.v.t, bt.table.cuda(), bt.dlens),
           lambda: rf.rf_paged_kv(bt.k.t, bt.v.t, bt.table.cuda().long(), bt.dlens, bt.ks, bt.vs),
           lambda: rf.rf_paged_kv(bt.k.t, bt.v.t[:1], bt.table.cuda(), bt.dlens, bt.ks, bt.vs)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(rf.RFError):
        rf.rf_attn_decode_paged(cache, o[:, :3].contiguous(), o[:, :3].contiguous(), 0.1, ws)
    with pytest.raises(rf.RFError):
        rf.rf_attn_decode_paged(cache, o, o, 0.1, None)
    assert rf.rf_get_device_status() == rf.RF_OK
