"""The paged-cache operators at sizes at which their kernels loop: lane groups
that take several heads in batches, CTAs that stay and take several pages and
heads, and offsets beyond 32 bits.  What a launch does with its sizes is
recomputed here from the device's SM count, so that each test asserts the path
it means.  Comparisons and tolerances are test_gpu_paged.py's."""
import numpy as np
import pytest
import torch

from oracle import paged as G
from tests.helpers import Guarded, to64
from tests.test_gpu_paged import BF16, F32, NR, Batch, _gen, assert_rows, attn_reference, \
    check_append, run_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_loop_gb300 as m
    assert torch.cuda.is_available()
    assert m.rf_get_device_status() == m.RF_OK
    return m


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def heads_per_group(rows, heads, d):
    """Heads a lane group takes one after the other, of rows = tokens x heads."""
    h, k = 1, 4
    while k < 2 * heads and rows * (d // 8) // k >= 1024 * sms():
        h, k = k, 2 * k
    return h


# ------------------------------------------------------------------ norm and rotation


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot,inter,norm", [(128, 128, False, True), (64, 32, True, True),
                                              (64, 64, False, False), (128, 0, False, True)])
@pytest.mark.parametrize("nh,Hq,Hkv", [(4, 9, 3), (4, 5, 2), (8, 9, 3), (16, 13, 1)])
def test_qk_norm_rope_several_heads_a_lane_group(rf, dtype, d, rot, inter, norm, nh, Hq, Hkv):
    """Blocks of heads that end early, batches of four behind one another, the next
    batch's loads before the present one's stores; in place, too."""
    T = -(-nh * 1024 * sms() // ((Hq + Hkv) * (d // 8))) + 5
    assert heads_per_group(T * (Hq + Hkv), max(Hq, Hkv), d) == nh
    nr = NR(rf, d, rot, inter, norm, dtype)
    g = _gen(T + d)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(dtype)
    pos = torch.randint(0, 600, (T,), generator=g, dtype=torch.int32)
    dev = qkv.cuda()
    qo, ko = Guarded((T, Hq, d), dtype), Guarded((T, Hkv, d), dtype)
    rf.rf_qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], qo.t, ko.t, nr.dev, pos.cuda())
    assert rf.rf_get_device_status() == rf.RF_OK
    assert_rows(qo.t, nr.ref(qkv[:, :Hq], pos, "q"), dtype, "q")
    assert_rows(ko.t, nr.ref(qkv[:, Hq:Hq + Hkv], pos, "k"), dtype, "k")
    qo.check("q")
    ko.check("k")
    rf.rf_qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, :Hq], dev[:, Hq:Hq + Hkv], nr.dev,
                       pos.cuda())
    assert torch.equal(dev[:, :Hq], qo.t) and torch.equal(dev[:, Hq:Hq + Hkv], ko.t)
    assert torch.equal(dev[:, Hq + Hkv:].cpu(), qkv[:, Hq + Hkv:])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_qk_norm_rope_tokens_far_apart(rf, dtype):
    """Tokens 2^31 + 8 elements apart."""
    nr = NR(rf, 64, 64, False, True, dtype)
    far = 2 ** 31 + 8
    raw = torch.empty(2 * far + 128, dtype=dtype, device="cuda")
    x = raw.as_strided((3, 2, 64), (far, 64, 1))
    src = torch.randn(3, 2, 64, generator=_gen(1)).to(dtype)
    x.copy_(src)
    pos = torch.arange(3, dtype=torch.int32)
    o = torch.empty(3, 2, 64, dtype=dtype, device="cuda")
    rf.rf_qk_norm_rope(x, None, o, None, nr.dev, pos.cuda())
    assert_rows(o, nr.ref(src, pos, "q"), dtype, "read far apart")
    rf.rf_qk_norm_rope(src.cuda(), None, x, None, nr.dev, pos.cuda())
    assert torch.equal(x, o)


# ------------------------------------------------------------------ append


def ragged(B, total, ps, seed):
    """(lengths, new tokens) of B sequences with `total` new ones: most begin inside a
    page, one is padding, one has no new tokens, one has a single one."""
    g = np.random.default_rng(seed)
    cut = np.sort(g.integers(0, total - 1, B - 4))
    new = np.diff(np.concatenate([[0], cut, [total - 1]])).tolist()
    new = [0] + new[:len(new) // 2] + [1, 0] + new[len(new) // 2:]
    start = g.integers(0, 5 * ps, len(new))
    lens = [int(s) + n for s, n in zip(start, new)]
    lens[0] = 0
    return lens, new


def run_prompts(rf, kind, ps, d, Hkv, Hq, B, total, rope, seed):
    lens, new = ragged(B, total, ps, seed)
    bt = Batch(kind, lens, Hkv, d, ps, seed=seed)
    cache = bt.device(rf)
    g = _gen(seed + 1)
    qkv = (torch.randn(total, Hq + 2 * Hkv, d, generator=g) *
           torch.exp(1.5 * torch.randn(total, Hq + 2 * Hkv, 1, generator=g))).to(BF16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    nr = NR(rf, d, rope[0], rope[1], rope[2], BF16, max_pos=max(lens), seed=seed)
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
    q_out = Guarded((total, Hq, d), BF16, fill=7.0)
    check_append(rf, bt, cache, new, k, v, nr, cu, q, q_out.t, f"{kind} {ps} {d} {total}")
    q_out.check("q_out")
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    assert_rows(q_out.t, nr.ref(q, pos, "q"), BF16, "q")


@pytest.mark.parametrize("d,nh,Hkv,Hq,ps,rope", [
    (128, 4, 5, 6, 64, (128, False, True)), (128, 8, 9, 4, 16, (64, True, True)),
    (64, 4, 5, 15, 32, (64, False, False)), (64, 8, 7, 7, 128, (64, True, True)),
    (64, 16, 9, 18, 64, (32, False, True)), (128, 4, 4, 1, 16, (128, True, False))])
def test_bf16_append_several_heads_a_lane_group(rf, d, nh, Hkv, Hq, ps, rope):
    total = -(-nh * 1024 * sms() // (2 * Hkv * (d // 8))) + 7
    assert heads_per_group(total * Hkv * 2, Hkv, d) == nh
    run_prompts(rf, "bf16", ps, d, Hkv, Hq, 23, total, rope, 900 + nh)


@pytest.mark.parametrize("ps,d,Hkv,rope", [
    (16, 64, 5, (64, False, True)), (16, 64, 7, (32, True, False)),          # 128 threads
    (32, 64, 5, (64, True, True)), (16, 128, 7, (128, False, True)),         # 256
    (64, 64, 7, (64, False, True)), (32, 128, 5, (64, False, False)),        # 512
    (64, 128, 5, (128, False, True)), (64, 128, 3, (128, True, True)),       # two sweeps of 512
    (128, 64, 7, (64, False, True)), (128, 64, 3, (48, True, True)),
    (128, 128, 3, (128, False, True)), (128, 128, 5, (96, True, False))])    # two sweeps of 1024
@pytest.mark.parametrize("Hq", [0, 6])
def test_e4m3_prompts_several_pages_and_heads_a_cta(rf, ps, d, Hkv, rope, Hq):
    """3.6 (page, head) pairs a CTA and more: ranges that begin and end inside a page's
    heads, pages that hold tokens of before and are rescaled."""
    pieces = ps * d // 8
    threads = pieces if pieces <= 512 else (512 if pieces <= 1024 else 1024)
    ctas = sms() * 1024 // threads
    B = 20
    total = int(3.6 * ctas / Hkv) * ps               # so many whole pages of new tokens
    if Hq:
        run_prompts(rf, "e4m3", ps, d, Hkv, Hq, B, total, rope, 920 + ps + d)
    else:                                            # no queries, no cu_seqlens
        n = total // 13
        assert n > 8 and 13 * (n // ps) * Hkv > 2 * ctas
        lens = [n + 11 * b for b in range(13)]
        bt = Batch("e4m3", lens, Hkv, d, ps, seed=940)
        cache = bt.device(rf)
        k, v = ((torch.randn(13 * n, Hkv, d, generator=_gen(941 + i)) *
                 torch.exp(1.5 * torch.randn(13 * n, Hkv, 1, generator=_gen(943 + i)))).to(BF16)
                for i in range(2))
        nr = NR(rf, d, rope[0], rope[1], rope[2], BF16, max_pos=max(lens))
        check_append(rf, bt, cache, [n] * 13, k, v, nr, None, what=f"uniform {ps} {d}")


# ------------------------------------------------------------------ offsets


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("new", [1, 5, 300])
def test_pages_beyond_32_bits(rf, kind, new):
    """A pool of 4.6e9 elements a tensor; the sequences live in its last pages."""
    num_pages, ps, d = 140000, 128, 128
    lens = [700, 310]
    bt = Batch(kind, lens, 2, d, ps, seed=950)
    base = num_pages - bt.num_pages
    e = kind == "e4m3"
    pages = [torch.zeros(num_pages, 2, ps, d, dtype=torch.uint8 if e else BF16, device="cuda")
             for _ in range(2)]
    scales = [torch.ones(num_pages, 2, device="cuda") if e else None for _ in range(2)]
    for t in range(2):
        pages[t][base:] = (torch.from_numpy(bt.pages[t]) if e else bt.pages[t]).cuda()
        if e:
            scales[t][base:] = torch.from_numpy(bt.scale[t]).cuda()
    dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = rf.rf_paged_kv(pages[0], pages[1], (bt.table + base).cuda(), dlens, *scales)
    q = torch.randn(2, 1, 8, d, generator=_gen(951)).to(BF16)
    got, status = run_attn(rf, bt, q, 0.0884, cache=cache)
    assert status == rf.RF_OK
    ref, tol = attn_reference(q, bt, 0.0884)
    assert (np.abs(to64(got) - ref) <= tol).all()
    k, v = (torch.randn(2 * new, 2, d, generator=_gen(952 + i)).to(BF16) for i in range(2))
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32).cuda() if new > 8 else None
    rf.rf_kv_append_paged(cache, k.cuda(), v.cuda(), None, cu)
    assert rf.rf_get_device_status() == rf.RF_OK
    k0, ks0 = bt.host(0)
    v0, vs0 = bt.host(1)
    want = G.append(k0, v0, ks0, vs0, bt.table.numpy(), lens, [new] * 2, k, v)
    for t in range(2):
        got = pages[t][base:].cpu()
        np.testing.assert_array_equal(got.numpy() if e else to64(got), want[t])
        if e:
            np.testing.assert_array_equal(scales[t][base:].cpu().numpy(), want[2 + t])
        assert not pages[t][:base].any()
