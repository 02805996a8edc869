"""Paged key-value cache on the GPU, through the public entry points, against
the plain 64-bit reference: append, decode and prompt attention."""
import math

import pytest
import torch

import gated_delta_rule_41_gb300 as kda
from paged_util import E4M3, check_attention, make_cache, ref_decode, ref_prefill

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_41_gb300 import build
    build.build()


def kv(c):
    return kda.KVPages(c["k"], c["v"], k_scale=c["ks"], v_scale=c["vs"])


def rand_q(rows, HQ, D, seed, amp=2.0):
    g = torch.Generator().manual_seed(seed)
    return (amp * torch.randn(rows, HQ, D, generator=g)).to(BF16).cuda()


def run_decode(lens, HQ, HKV, D, page, dtype, window=0, sinks=0, layout="rows", seed=1, amp=2.0,
               scale=None):
    c = make_cache(lens, page, HKV, D, dtype, seed, layout)
    q = rand_q(len(lens), HQ, D, seed + 100, amp)
    o, lse = kda.paged_decode(q, kv(c), c["table"], c["lens"], scale=scale, window=window,
                              sinks=sinks, return_lse=True)
    kda.check()
    check_attention(o, lse, ref_decode(q, c, D ** -0.5 if scale is None else scale, window, sinks))
    return q, c, o, lse


# ---- decode ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_lengths(page, D, dtype):
    """Idle rows, one token, page ends and their neighbours, several pages."""
    run_decode([0, 1, 2, 15, 16, 17, page - 1, page, page + 1, 3 * page + 5, 700], 4, 2, D, page,
               dtype)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("HQ,HKV", [(1, 1), (3, 3), (2, 1), (6, 2), (5, 1), (16, 2), (20, 2),
                                    (16, 1), (24, 1), (64, 1)])
def test_decode_heads(HQ, HKV, dtype):
    run_decode([300, 1, 77], HQ, HKV, 128, 32, dtype, seed=2)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (40, 4), (100, 70), (300, 4),
                                          (5000, 9), (64, 1000)])
def test_decode_window(window, sinks, dtype):
    run_decode([0, 1, 39, 40, 41, 45, 128, 500, 1111], 8, 2, 64, 16, dtype, window, sinks, seed=3)


@pytest.mark.parametrize("layout", ["rows", "heads", "joint"])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_decode_layouts(layout, dtype):
    run_decode([100, 33, 257], 8, 4, 128, 32, dtype, layout=layout, seed=4)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens", [[70001], [9000, 12, 30000], [2500] * 40, [4096, 1] * 70])
def test_decode_long_and_many(lens, dtype):
    """One long row, unequal ones, and more rows than the GPU has room for."""
    run_decode(lens, 8, 2, 64, 64, dtype, seed=5)


@pytest.mark.parametrize("amp,scale", [(60.0, 1.0), (0.0, None), (1e4, 0.125), (2.0, 0.0),
                                       (2.0, -0.3)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_decode_logits_of_any_size(amp, scale, dtype):
    """Weights that are all but one-hot, all equal, and a falling scale."""
    run_decode([513, 90, 16], 4, 1, 128, 16, dtype, seed=6, amp=amp, scale=scale)


def test_decode_strided_q_out_workspace_and_stream():
    c = make_cache([130, 999, 5], 32, 2, 128, BF16, 7)
    wide = rand_q(3, 12, 128, 8)
    q = wide[:, 2:10]
    pages = kv(c)
    ref = kda.paged_decode(q.contiguous(), pages, c["table"], c["lens"])
    ws = kda.paged_decode_workspace(pages, 3, 8)
    out = torch.full((3, 8, 128), 7.0, dtype=BF16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.paged_decode(q, pages, c["table"], c["lens"], out=out, workspace=ws, stream=s)
    fresh = kda.paged_decode(q, pages, c["table"], c["lens"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert got is out
    assert torch.equal(out, ref) and torch.equal(fresh, ref)


def test_decode_repeats_bit_for_bit():
    c = make_cache([7000, 3, 1234] * 9, 64, 2, 128, BF16, 9)
    q = rand_q(27, 16, 128, 10)
    a = kda.paged_decode(q, kv(c), c["table"], c["lens"], return_lse=True)
    for _ in range(5):
        b = kda.paged_decode(q, kv(c), c["table"], c["lens"], return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_in_a_graph():
    c = make_cache([500, 20], 32, 2, 128, BF16, 11)
    q = rand_q(2, 8, 128, 12)
    pages = kv(c)
    ref = kda.paged_decode(q, pages, c["table"], c["lens"])
    ws = kda.paged_decode_workspace(pages, 2, 8)
    out = torch.zeros_like(ref)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.paged_decode(q, pages, c["table"], c["lens"], out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_decode_large_offsets():
    """Pages past 2^31 elements of the pool."""
    page, HKV, D = 256, 8, 128
    n = (1 << 31) // (page * HKV * D) + 20
    k = torch.empty(n, page, HKV, D, dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    table = torch.arange(n - 3, n, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    g = torch.Generator().manual_seed(13)
    for t in (k, v):
        t[n - 3:] = torch.randn(3, page, HKV, D, generator=g).to(BF16).cuda()
    lens = torch.tensor([600], dtype=torch.int32, device="cuda")
    q = rand_q(1, 16, D, 14)
    tail = dict(k=k[n - 3:], v=v[n - 3:], ks=None, vs=None, table=table - (n - 3), lens=lens)
    o, lse = kda.paged_decode(q, kda.KVPages(k, v), table, lens, return_lse=True)
    check_attention(o, lse, ref_decode(q, tail, D ** -0.5))
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    q2 = rand_q(2, 16, D, 15)
    o, lse = kda.paged_prefill(q2, kda.KVPages(k, v), table, lens, cu, return_lse=True)
    check_attention(o, lse, ref_prefill(q2, tail, [2], D ** -0.5))
    kda.check()


@pytest.mark.parametrize("prefill", [False, True])
def test_bad_tables_are_reported_and_harmless(prefill):
    """Lengths that the table cannot hold count as 0; tokens of pages out of
    range count as zeros; other rows are not affected."""
    c = make_cache([40, 40, 40], 16, 1, 64, BF16, 16, poison=False)
    q = rand_q(3, 2, 64, 17)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")

    def call(table, lens):
        if prefill:
            return kda.paged_prefill(q, kv(c), table, lens, cu, return_lse=True)
        return kda.paged_decode(q, kv(c), table, lens, return_lse=True)

    good, _ = call(c["table"], c["lens"])
    for bad in (-5, 10 ** 6):
        lens = c["lens"].clone()
        lens[1] = bad
        o, lse = call(c["table"], lens)
        with pytest.raises(kda.KdaError) as e:
            kda.check()
        assert e.value.status == 2
        assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    for bad in (-1, 10 ** 6):
        table = c["table"].clone()
        table[1, 1] = bad
        o, _ = call(table, c["lens"])
        with pytest.raises(kda.KdaError) as e:
            kda.check()
        assert e.value.status == 2
        zeroed = dict(c, k=c["k"].clone(), v=c["v"].clone())
        zeroed["k"][c["table"][1, 1].item()] = 0
        zeroed["v"][c["table"][1, 1].item()] = 0
        c2 = dict(zeroed)
        want, _ = (kda.paged_prefill(q, kv(c2), c["table"], c["lens"], cu, return_lse=True)
                   if prefill else
                   kda.paged_decode(q, kv(c2), c["table"], c["lens"], return_lse=True))
        assert torch.equal(o[1], want[1]) and torch.equal(o[0], good[0])
    kda.check()


# ---- prompts ----

def run_prefill(lens, qn, HQ, HKV, D, page, dtype, window=0, sinks=0, layout="rows", seed=1,
                amp=2.0, scale=None):
    c = make_cache(lens, page, HKV, D, dtype, seed, layout)
    q = rand_q(sum(qn), HQ, D, seed + 100, amp)
    cu = torch.tensor([0] + qn).cumsum(0).to(torch.int32).cuda()
    o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, scale=scale, window=window,
                               sinks=sinks, return_lse=True)
    kda.check()
    check_attention(o, lse, ref_prefill(q, c, qn, D ** -0.5 if scale is None else scale, window,
                                        sinks))
    return q, c, cu, o, lse


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_prefill_lengths(page, D, dtype):
    """Empty prompts, one token, tile and page ends, prompts in chunks."""
    qn = [1, 0, 2, 63, 64, 65, 127, 129, 300, 5, 1]
    lens = [1, 0, 2, 63, 64, 65, 127, 129, 300, 400, 257]
    run_prefill(lens, qn, 4, 2, D, page, dtype)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("HQ,HKV", [(1, 1), (3, 3), (2, 1), (6, 2), (5, 1), (7, 1), (16, 2),
                                    (16, 1), (24, 1), (33, 1), (64, 1)])
def test_prefill_heads(HQ, HKV, dtype):
    run_prefill([150, 90], [150, 40], HQ, HKV, 128, 32, dtype, seed=2)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (40, 4), (128, 130), (300, 4),
                                          (5000, 9), (64, 1000)])
def test_prefill_window(window, sinks, dtype):
    run_prefill([700, 41, 1500], [700, 41, 100], 4, 2, 64, 16, dtype, window, sinks, seed=3)


@pytest.mark.parametrize("layout", ["rows", "heads", "joint"])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_prefill_layouts(layout, dtype):
    run_prefill([260, 33], [200, 33], 8, 4, 128, 32, dtype, layout=layout, seed=4)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,qn", [([20000], [3]), ([5000, 9000], [17, 130]), ([2500], [2500]),
                                     ([130] * 40, [130] * 40)])
def test_prefill_few_rows_and_many(lens, qn, dtype):
    """A few queries over a long context, long prompts, many prompts."""
    run_prefill(lens, qn, 4, 2, 64, 64, dtype, seed=5)


@pytest.mark.parametrize("amp,scale", [(60.0, 1.0), (0.0, None), (1e4, 0.125), (2.0, 0.0),
                                       (2.0, -0.3)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_prefill_logits_of_any_size(amp, scale, dtype):
    run_prefill([400, 90], [300, 90], 4, 1, 128, 16, dtype, seed=6, amp=amp, scale=scale)


def test_prefill_more_queries_than_tokens():
    """Queries at negative positions see nothing."""
    run_prefill([10, 0, 100], [30, 4, 150], 4, 2, 64, 16, BF16, seed=7)


def test_prefill_matches_decode():
    q, c, cu, o, lse = run_prefill([333, 64], [1, 1], 8, 2, 128, 32, BF16, seed=8)
    d, dl = kda.paged_decode(q, kv(c), c["table"], c["lens"], return_lse=True)
    assert (o.float() - d.float()).abs().max() <= 2.0 ** -7 * d.float().abs().max()
    assert (lse - dl).abs().max() < 1e-4


def test_prefill_strided_q_out_workspace_and_stream():
    c = make_cache([300, 50], 32, 2, 128, BF16, 9)
    wide = rand_q(350, 12, 128, 10)
    q = wide[:, 2:10]
    cu = torch.tensor([0, 300, 350], dtype=torch.int32, device="cuda")
    pages = kv(c)
    ref = kda.paged_prefill(q.contiguous(), pages, c["table"], c["lens"], cu)
    ws = kda.paged_prefill_workspace(pages, 2, 350, 8)
    out = torch.full((350, 8, 128), 7.0, dtype=BF16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kda.paged_prefill(q, pages, c["table"], c["lens"], cu, out=out, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, ref)
    again = kda.paged_prefill(q, pages, c["table"], c["lens"], cu)
    assert torch.equal(again, ref)


@pytest.mark.parametrize("cu", [[0, 30, 20, 50], [0, 10, 20, 40], [1, 10, 20, 50],
                                [-3, 10, 20, 50]])
def test_bad_cu_seqlens_leave_no_effect(cu):
    c = make_cache([50, 50, 50], 16, 1, 64, BF16, 11, poison=False)
    q = rand_q(50, 2, 64, 12)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, out=out)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2 and (out == 3).all()
    before = c["k"].clone(), c["v"].clone()
    kda.paged_append(kv(c), q[:, :1], q[:, 1:], c["table"], c["lens"], cu)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2
    assert torch.equal(before[0], c["k"]) and torch.equal(before[1], c["v"])


# ---- append ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["rows", "heads", "joint"])
@pytest.mark.parametrize("packed", [False, True])
def test_append(packed, layout, D, dtype):
    """Codes and rows are exact: K and V land where the table says, and no
    other slot changes."""
    lens, HKV, page = [5, 0, 16, 17, 200, 33], 3, 16
    qn = [5, 0, 3, 17, 70, 40] if packed else [1] * 6      # 40 > 33: seven are dropped
    c = make_cache(lens, page, HKV, D, dtype, 20, layout, poison=False)
    T = sum(qn)
    g = torch.Generator().manual_seed(21)
    qkv = torch.randn(T, 2 * HKV + 1, D, generator=g).to(BF16)
    qkv[0, :, 0], qkv[0, :, 1], qkv[0, :, 2] = math.inf, -math.inf, 3e38
    qkv = qkv.cuda()
    nk, nv = qkv[:, :HKV], qkv[:, HKV:2 * HKV]
    want = []
    for pool, new, sc in ((c["k"], nk, c["ks"]), (c["v"], nv, c["vs"])):
        w, at = pool.clone(), 0
        raw = w.view(torch.uint8) if dtype == E4M3 else w
        x = new
        if dtype == E4M3:
            x = (new.float() * (1.0 / sc)[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        for s, n in enumerate(qn):
            for i in range(n):
                pos = lens[s] - n + i
                if pos >= 0:
                    raw[c["table"][s, pos // page].item(), pos % page] = x[at]
                at += 1
        want.append(raw)
    cu = torch.tensor([0] + qn).cumsum(0).to(torch.int32).cuda() if packed else None
    kda.paged_append(kv(c), nk, nv, c["table"], c["lens"], cu)
    kda.check()
    for pool, w in zip((c["k"], c["v"]), want):
        assert torch.equal(pool.view(torch.uint8) if dtype == E4M3 else pool, w)


def test_append_nan_and_missing_scales():
    c = make_cache([2, 1], 16, 1, 64, E4M3, 22, poison=False)
    x = torch.full((2, 1, 64), 3.3, dtype=BF16, device="cuda")
    x[0, 0, 5] = math.nan
    kda.paged_append(kda.KVPages(c["k"], c["v"]), x, x, c["table"], c["lens"])
    got = c["k"].view(torch.uint8)[c["table"][0, 0].item(), 1, 0].view(E4M3).float()
    assert got[5].isnan() and (got[:5] == 3.25).all()


def test_append_bad_page_drops_the_write():
    c = make_cache([3, 4], 16, 1, 64, BF16, 23, poison=False)
    before = c["k"].clone()
    c["table"][:, 0] = torch.tensor([-1, 10 ** 6], dtype=torch.int32)
    x = torch.ones(2, 1, 64, dtype=BF16, device="cuda")
    kda.paged_append(kv(c), x, x, c["table"], c["lens"])
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2 and torch.equal(before, c["k"])


# ---- refusals ----

def test_refusals():
    c = make_cache([40, 20], 16, 2, 64, BF16, 30)
    pages, q = kv(c), rand_q(2, 4, 64, 31)
    t, n = c["table"], c["lens"]

    def status(fn):
        with pytest.raises(kda.KdaError) as e:
            fn()
        return e.value.status

    assert status(lambda: kda.paged_decode(q.float(), pages, t, n)) == 3
    assert status(lambda: kda.paged_decode(q[:, :3].contiguous(), pages, t, n)) == 2
    assert status(lambda: kda.paged_decode(q[..., :32], pages, t, n)) == 1
    assert status(lambda: kda.paged_decode(q, pages, t.long(), n)) == 1
    assert status(lambda: kda.paged_decode(q, pages, t, n[:1])) == 1
    assert status(lambda: kda.paged_decode(q, pages, t[:1], n[:1])) == 2
    assert status(lambda: kda.paged_decode(q, pages, t, n, window=-1)) == 1
    assert status(lambda: kda.paged_decode(q, pages, t, n, scale=math.nan)) == 1
    assert status(lambda: kda.paged_decode(q, pages, t, n, out=q.float())) == 1
    assert status(lambda: kda.paged_decode(rand_q(2, 130, 64, 1), pages, t, n)) == 3
    f32 = kda.KVPages(c["k"].float(), c["v"].float())
    assert status(lambda: kda.paged_decode(q, f32, t, n)) == 3
    odd = kda.KVPages(c["k"][:, :10], c["v"][:, :10])
    assert status(lambda: kda.paged_decode(q, odd, t, n)) == 3
    assert status(lambda: kda.KVPages(c["k"], c["v"][:2])) == 1
    assert status(lambda: kda.KVPages(c["k"], c["v"], k_scale=torch.ones(2).cuda())) == 1
    assert status(lambda: kda.KVPages(c["k"].half(), c["v"].half())) == 3
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    assert status(lambda: kda.paged_prefill(q, pages, t, n, cu[:2])) == 1
    assert status(lambda: kda.paged_append(pages, q, q, t, n)) == 1
    assert status(lambda: kda.paged_append(pages, q[:1, :2], q[:1, :2], t, n)) == 2
    assert kda.paged_prefill(q[:0], pages, t, n, cu).shape == (0, 4, 64)
    kda.check()


# ---- values of any size, repeats ----

@pytest.mark.parametrize("case", ["tiny", "huge", "zeros_first", "outliers", "infinite"])
@pytest.mark.parametrize("prefill", [False, True])
def test_values_of_any_size(prefill, case):
    """V scaled as a whole, a first tile of zeros, a few tokens a million times
    larger than the others, and infinities that only later queries see."""
    lens, qn = [700], [300]
    c = make_cache(lens, 32, 2, 128, BF16, 40)
    page = lambda j: c["table"][0, j // 32].item()
    if case == "tiny":
        c["v"].mul_(2.0 ** -60)
    elif case == "huge":
        c["v"].mul_(2.0 ** 60)
    elif case == "zeros_first":
        for j in range(0, 160, 32):
            c["v"][page(j)] = 0
    elif case == "outliers":
        for j in (130, 450, 690):
            c["v"][page(j), j % 32] *= 2.0 ** 20
    else:
        c["v"][page(650), 650 % 32, :, 3] = math.inf
    if prefill:
        q = rand_q(300, 4, 128, 41)
        cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
        o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, return_lse=True)
        ref = ref_prefill(q, c, qn, 128 ** -0.5)
    else:
        q = rand_q(1, 4, 128, 41)
        o, lse = kda.paged_decode(q, kv(c), c["table"], c["lens"], return_lse=True)
        ref = ref_decode(q, c, 128 ** -0.5)
    kda.check()
    if case == "infinite":
        # queries behind the infinity, and the other channels, are as ever
        other = [d for d in range(128) if d != 3]
        sees = torch.tensor([j >= 650 for j in range(400, 700)] if prefill else [True])
        assert not torch.isfinite(o[sees.cuda()][..., 3]).any()
        keep = ~sees
        ref = [x[..., other] if x.dim() == 3 else x for x in ref]
        check_attention(o[..., other][keep.cuda()], lse[keep.cuda()], [x[keep] for x in ref])
    else:
        check_attention(o, lse, ref)


@pytest.mark.parametrize("amp", [1e8, 1e16, 1e25, 1e37])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_logits_beyond_single_precision(amp, dtype):
    """Logits so large that their rounding errors exceed any weight: the calls
    end, and every output is a mean of values."""
    c = make_cache([400, 200], 32, 1, 128, dtype, 47)
    q = rand_q(300, 5, 128, 48, amp)
    cu = torch.tensor([0, 200, 300], dtype=torch.int32, device="cuda")
    o, _ = kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, scale=1.0, return_lse=True)
    d, _ = kda.paged_decode(q[:2], kv(c), c["table"], c["lens"], scale=1.0, return_lse=True)
    kda.check()
    for x in (o, d) if amp < 1e36 else ():
        assert torch.isfinite(x).all() and x.abs().max() < 20


@pytest.mark.parametrize("lens,qn", [([9000], [5]), ([3000, 500, 40], [3000, 77, 40])])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_prefill_repeats_bit_for_bit(lens, qn, dtype):
    q, c, cu, o, lse = run_prefill(lens, qn, 6, 2, 128, 64, dtype, seed=42)
    for _ in range(4):
        b = kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, return_lse=True)
        assert torch.equal(o, b[0]) and torch.equal(lse, b[1])


def test_decode_workspace_serves_calls_of_any_sizes():
    """One workspace through calls of other batches and lengths, in turn."""
    a = make_cache([5000, 1, 800], 64, 2, 128, BF16, 43)
    b = make_cache([60] * 33 + [20000], 64, 2, 128, BF16, 44)
    qa, qb = rand_q(3, 8, 128, 45), rand_q(34, 8, 128, 46)
    pa, pb = kv(a), kv(b)
    ws = kda.paged_decode_workspace(pa, 3, 8)
    want = (kda.paged_decode(qa, pa, a["table"], a["lens"]),
            kda.paged_decode(qb, pb, b["table"], b["lens"]))
    for _ in range(3):
        got = (kda.paged_decode(qa, pa, a["table"], a["lens"], workspace=ws),
               kda.paged_decode(qb, pb, b["table"], b["lens"], workspace=ws))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
