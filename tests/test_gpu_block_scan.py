"""The gated linear recurrence on the GPU against the token-by-token 64-bit reference: forward,
backward, packed sequences, the single-token step."""
import pytest
import torch

import gated_delta_rule_41_gb300 as kda
from block_util import BF16, F32, check, d64, ref_scan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_41_gb300 import build
    build.build()


def make(B, T, C, dtype, seed, rows, mu=-3.0, sigma=1.5, slices=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, g = r(B, T, C), -torch.exp(sigma * r(B, T, C) + mu)
    x, g, do = x.to(dtype).cuda(), g.to(dtype).cuda(), r(B, T, C).to(dtype).cuda()
    if slices:
        wide = torch.full((B, T, 3 * C + 16), float("nan"), dtype=dtype, device="cuda")
        wide[..., :C], wide[..., 2 * C + 8:3 * C + 8] = x, g
        x, g = wide[..., :C], wide[..., 2 * C + 8:3 * C + 8]
    return x, g, do, r(rows, C).cuda(), r(rows, C).cuda()


def run(x, g, do, h0, dht, tied=False, cu=None, keep=True):
    dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, ht, saved = kda.gated_scan_fwd(x, g, h0, output_final_state=True, tied=tied, cu_seqlens=dev,
                                      save_for_backward=True)
    grads = kda.gated_scan_bwd(x, g, do, saved if keep else None, dht=dht, initial_state=h0, tied=tied,
                               cu_seqlens=dev)
    kda.check()
    ref = ref_scan(x, g, h0, tied, cu, do, dht)
    got = dict(grads, o=o, ht=ht)
    for n, t in got.items():
        if t is not None:
            check(n, t, ref[n], ref[n + "~"])
    return got


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(T, dtype, tied):
    run(*make(2, T, 72, dtype, T, 2), tied=tied)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [1, 2, 3, 7, 8, 31, 62, 63, 64, 65, 66, 72, 100, 127, 128, 130, 200, 1000])
def test_widths(C, dtype):
    run(*make(1, 150, C, dtype, C, 1), tied=C % 2 == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,C", [(1, 5000, 64), (1, 3000, 40), (3, 1000, 256), (5, 700, 640), (2, 2100, 1024)])
def test_long(B, T, C, dtype):
    """Axes of many tiles, with few channels (several CTAs on one axis) and with many."""
    run(*make(B, T, C, dtype, 7, B, mu=-5.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slices_and_no_states(dtype):
    x, g, do, h0, dht = make(2, 200, 48, dtype, 3, 2, slices=True)
    run(x, g, do, h0, dht, tied=True)
    run(x, g, do, None, None)
    run(x, g, do, h0, None, keep=False)
    x, g, do, h0, dht = make(2, 90, 33, dtype, 4, 2, slices=True)
    run(x, g, do, h0, dht)


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", [[0, 1], [0, 130], [0, 1, 2, 3], [0, 64, 128, 192], [0, 0, 5, 5, 5, 130, 130],
                                [0, 63, 64, 65, 127, 128, 129, 300], [0, 16, 31, 32, 160, 400], [0, 0, 0, 7],
                                list(range(0, 140)) + [300]])
def test_packed(cu, dtype, tied):
    x, g, do, h0, dht = make(1, cu[-1], 72, dtype, len(cu), len(cu) - 1)
    run(x, g, do, h0, dht, tied=tied, cu=cu)
    run(x, g, do, None, None, tied=tied, cu=cu, keep=False)


def test_packed_long():
    cu = [0, 900, 900, 1000, 4096, 4097, 6000]
    run(*make(1, 6000, 64, BF16, 5, 6, mu=-5.0), cu=cu)
    run(*make(1, 6000, 136, F32, 5, 6, mu=-5.0), cu=cu)


def test_packed_is_each_alone():
    """One of several packed sequences, within the two orders' roundings, is that sequence alone;
    what is not finite in one does not reach its neighbours."""
    cu = [0, 100, 300, 333]
    x, g, do, h0, dht = make(1, 333, 64, F32, 9, 3)
    x[0, 50], x[0, 310, 3], h0[0, 5] = float("inf"), float("nan"), float("nan")
    dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, ht, saved = kda.gated_scan_fwd(x, g, h0, True, cu_seqlens=dev, save_for_backward=True)
    gr = kda.gated_scan_bwd(x, g, do, saved, dht=dht, initial_state=h0, cu_seqlens=dev)
    ref = ref_scan(x[:, 100:300], g[:, 100:300], h0[1:2], do=do[:, 100:300], dht=dht[1:2])
    for n, t in (("o", o), ("dx", gr["dx"]), ("dg", gr["dg"])):
        check(n, t[:, 100:300], ref[n], ref[n + "~"])
    check("ht", ht[1:2], ref["ht"], ref["ht~"])
    check("dh0", gr["dh0"][1:2], ref["dh0"], ref["dh0~"])
    assert torch.isnan(o[0, :, 5][:100]).all() and torch.isfinite(o[0, :50, 4]).all()


@pytest.mark.parametrize("cu", [[1, 50, 100], [0, 60, 50, 100], [0, 50, 99], [0, 50, 101], [0, -1, 100],
                                [0, 2000000000, 100]])
def test_bad_cu_seqlens(cu):
    """Reported; the final states are the initial ones, nothing else is written."""
    x, g, do, h0, dht = make(1, 100, 72, BF16, 1, len(cu) - 1)
    dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full_like(x, 7.0)
    _, ht, saved = kda.gated_scan_fwd(x, g, h0, True, cu_seqlens=dev, out=o, save_for_backward=True)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2
    assert (o == 7).all() and torch.equal(ht, h0)
    grads = dict(dx=torch.full_like(x, 7.0), dg=torch.full_like(x, 7.0), dh0=torch.zeros_like(h0))
    kda.gated_scan_bwd(x, g, do, torch.zeros_like(saved), dht=dht, initial_state=h0, cu_seqlens=dev, grads=grads)
    with pytest.raises(kda.KdaError):
        kda.check()
    assert (grads["dx"] == 7).all() and (grads["dg"] == 7).all() and torch.equal(grads["dh0"], dht)
    kda.check()


def test_empty():
    x, g, do, h0, dht = make(3, 0, 40, F32, 1, 3)
    o, ht, saved = kda.gated_scan_fwd(x, g, h0, True, save_for_backward=True)
    gr = kda.gated_scan_bwd(x, g, do, saved, dht=dht, initial_state=h0)
    assert o.shape == (3, 0, 40) and torch.equal(ht, h0) and torch.equal(gr["dh0"], dht)
    _, ht = kda.gated_scan_fwd(x, g, None, True)
    assert (ht == 0).all()
    cu = torch.zeros(5, dtype=torch.int32, device="cuda")
    h0 = torch.randn(4, 40, device="cuda")
    assert torch.equal(kda.gated_scan_fwd(x[:1], g[:1], h0, True, cu_seqlens=cu)[1], h0)
    o, ht = kda.gated_scan_fwd(x[:0], g[:0], None, True)
    assert ht.shape == (0, 40)
    kda.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates_of_any_size(dtype):
    """No decay at all, decays that act over the whole axis, decays that forget at once, and
    small inputs behind a large state that a strong decay removes."""
    B, T, C = 1, 400, 64
    x, g, do, h0, dht = make(B, T, C, dtype, 2, B)
    g[..., 0::8] = 0.0
    g[..., 1::8] = -1e-4
    g[..., 2::8] = -200.0
    g[..., 3::8] = -float("inf")
    g[..., 4::8] = -0.25
    g[..., 5::8] = -30.0
    h0 *= 1e6
    run(x, g, do, h0, dht)
    run(x, g, do, h0, dht, tied=True)
    g[..., 6::8] = 0.01                     # growth
    run(x[:, :60], g[:, :60], do[:, :60].contiguous(), h0, dht)


def test_nan_stays_in_its_channel():
    x, g, do, h0, dht = make(1, 300, 72, F32, 2, 1)
    x[0, 100, 5], g[0, 200, 9] = float("nan"), float("nan")
    o, ht = kda.gated_scan_fwd(x, g, h0, True)
    bad = torch.isnan(o[0])
    assert bad[100:, 5].all() and bad[200:, 9].all()
    bad[:, 5] = bad[:, 9] = False
    assert not bad.any() and not torch.isnan(o[0, :100, 5]).any()


def test_gradients_are_differences():
    """Central differences of the 64-bit forward (the gradients of the reference itself)."""
    gen = torch.Generator().manual_seed(3)
    x, h0, w, wt = (torch.randn(*s, generator=gen).double() for s in ((1, 9, 3), (1, 3), (1, 9, 3), (1, 3)))
    g = -torch.rand(1, 9, 3, generator=gen).double()
    for tied in (False, True):
        def loss(x, g, h0):
            r = ref_scan(x, g, h0, tied)
            return (r["o"] * w).sum() + (r["ht"] * wt).sum()
        ref = ref_scan(x, g, h0, tied, do=w, dht=wt)
        for n, t in (("dx", x), ("dg", g), ("dh0", h0)):
            num = torch.zeros_like(t)
            for i in range(t.numel()):
                d = torch.zeros_like(t)
                d.view(-1)[i] = 1e-5
                args = [v + d if v is t else v for v in (x, g, h0)], [v - d if v is t else v for v in (x, g, h0)]
                num.view(-1)[i] = (loss(*args[0]) - loss(*args[1])) / 2e-5
            assert torch.allclose(num, ref[n], atol=1e-8), n


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,C", [(1, 1), (1, 64), (3, 77), (5, 256), (300, 1000)])
def test_step(B, C, dtype, tied):
    gen = torch.Generator().manual_seed(B + C)
    wide = torch.randn(B, 2 * C + 8, generator=gen).to(dtype).cuda()
    x, g = wide[:, :C], -wide[:, C + 8:].abs()
    h0 = torch.randn(B, C, generator=gen).cuda()
    ref = ref_scan(x[:, None], g[:, None], h0, tied)
    nxt, old = torch.empty_like(h0), h0.clone()
    o = kda.gated_scan_step(x, g, h0, tied=tied, new_state=nxt)
    assert torch.equal(h0, old)
    check("o", o, ref["o"][:, 0], ref["o~"][:, 0])
    check("state", nxt, ref["ht"], ref["ht~"])
    o2 = kda.gated_scan_step(x, g, h0, tied=tied)
    assert torch.equal(o, o2) and torch.equal(h0, nxt)


def test_steps_are_the_scan():
    x, g, _, h0, _ = make(4, 40, 96, BF16, 6, 4)
    o, ht = kda.gated_scan_fwd(x, g, h0, True)
    h = h0.clone()
    steps = torch.stack([kda.gated_scan_step(x[:, t], g[:, t], h) for t in range(40)], 1)
    ref = ref_scan(x, g, h0)
    check("o", o, ref["o"], ref["o~"])
    check("steps", steps, ref["o"], ref["o~"])
    check("ht", h, ref["ht"], ref["ht~"])


def test_chained_halves():
    """Two halves with the state handed on are the whole."""
    x, g, do, h0, dht = make(2, 500, 64, F32, 8, 2)
    ref = ref_scan(x, g, h0, do=do, dht=dht)
    o1, h1 = kda.gated_scan_fwd(x[:, :170], g[:, :170], h0, True)
    o2, h2 = kda.gated_scan_fwd(x[:, 170:], g[:, 170:], h1, True)
    check("o", torch.cat([o1, o2], 1), ref["o"], 2 * ref["o~"])
    check("ht", h2, ref["ht"], 2 * ref["ht~"])
    b = kda.gated_scan_bwd(x[:, 170:], g[:, 170:], do[:, 170:].contiguous(), dht=dht, initial_state=h1)
    a = kda.gated_scan_bwd(x[:, :170], g[:, :170], do[:, :170].contiguous(), dht=b["dh0"], initial_state=h0)
    check("dg", torch.cat([a["dg"], b["dg"]], 1), ref["dg"], 2 * ref["dg~"])
    check("dh0", a["dh0"], ref["dh0"], 2 * ref["dh0~"])


@pytest.mark.parametrize("cu", [None, [0, 300, 1500, 2000]])
def test_same_bits_in_graphs_and_on_streams(cu):
    """The same call gives the same bits: again, in a replayed graph, and on another stream beside
    another call."""
    x, g, do, h0, dht = make(1, 2000, 128, BF16, 4, 1 if cu is None else 3)
    dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")

    def both(stream=None):
        o, ht, sv = kda.gated_scan_fwd(x, g, h0, True, cu_seqlens=dev, save_for_backward=True, stream=stream)
        gr = kda.gated_scan_bwd(x, g, do, sv, dht=dht, initial_state=h0, cu_seqlens=dev, stream=stream)
        return o, ht, gr["dx"], gr["dg"], gr["dh0"]

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    others, here = both(side), both()
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(want, others, here):
        assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.zero_()
    graph.replay()
    graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    kda.check()


def test_offsets_past_32_bits():
    """Rows that lie beyond 2^31 elements from their tensor's start."""
    T, C, far = 3, 64, 3 << 29
    big = torch.empty((T - 1) * far + C, dtype=BF16, device="cuda")
    x = big.as_strided((1, T, C), (T * far, far, 1))
    v, g, do, h0, dht = make(1, T, C, BF16, 4, 1)
    x.copy_(v)
    want, got = kda.gated_scan_fwd(v, g, h0)[0], kda.gated_scan_fwd(x, g, h0)[0]
    assert torch.equal(want, got)
    a, b = (kda.gated_scan_bwd(t, g, do, initial_state=h0, tied=True) for t in (v, x))
    assert torch.equal(a["dg"], b["dg"]) and torch.equal(a["dx"], b["dx"])


def test_refusals():
    x, g, do, h0, dht = make(2, 20, 16, BF16, 1, 2)

    def refused(status, f, *a, **k):
        with pytest.raises(kda.KdaError) as e:
            f(*a, **k)
        assert e.value.status == status

    refused(1, kda.gated_scan_fwd, x, g.float())
    refused(3, kda.gated_scan_fwd, x.half(), g.half())
    refused(1, kda.gated_scan_fwd, x, g[:, :10])
    refused(1, kda.gated_scan_fwd, x.transpose(1, 2), g.transpose(1, 2))
    refused(1, kda.gated_scan_fwd, x.cpu(), g)
    refused(1, kda.gated_scan_fwd, x, g, h0[:1])
    refused(1, kda.gated_scan_fwd, x, g, h0.bfloat16())
    refused(2, kda.gated_scan_fwd, x, g, cu_seqlens=torch.tensor([0, 20], dtype=torch.int32, device="cuda"))
    refused(1, kda.gated_scan_fwd, x[:1], g[:1], cu_seqlens=torch.tensor([0, 20], device="cuda"))
    refused(2, kda.gated_scan_fwd, x[:, :1].expand(2, 20, 16), g)
    refused(1, kda.gated_scan_bwd, x, g, do.float())
    refused(1, kda.gated_scan_bwd, x, g, do, saved=h0)
    refused(1, kda.gated_scan_step, x[:, 0], g[:, 0], h0[:1])
    kda.check()


def exchange(ctas, turns, slow_cta=-1, slow_turn=0, stall=0, limit=2_000_000_000):
    """What each CTA sums up over the turns."""
    from gated_delta_rule_41_gb300 import block
    sums = torch.zeros(ctas, device="cuda")
    assert block._lib().kda_selftest_exchange(ctas, turns, slow_cta, slow_turn, stall, limit, sums.data_ptr(),
                                              torch.cuda.current_stream().cuda_stream) == 0
    return sums.tolist()


def summed(ctas, turns):
    return [float(turns * (turns + 1) // 2 * (ctas * (ctas + 1) // 2))] * ctas


@pytest.mark.parametrize("ctas", [1, 2, 5, 8, 13, 16])
def test_exchange_of_a_cluster(ctas):
    for turns in (1, 2, 7, 100):
        assert exchange(ctas, turns) == summed(ctas, turns)
        assert exchange(ctas, turns, ctas // 2, turns // 2, 1_000_000) == summed(ctas, turns)
    kda.check()


@pytest.mark.parametrize("ctas", [2, 5, 13])
@pytest.mark.parametrize("turns,slow_turn", [(1, 0), (2, 0), (9, 0), (9, 3), (9, 7), (9, 8), (200, 100)])
def test_a_wait_that_gives_up(ctas, turns, slow_turn):
    """A CTA stalls for 5 ms in one turn and the others' waits run out after 0.1 ms: that is reported, all CTAs
    end, and what runs next is right."""
    kda.check()
    got = exchange(ctas, turns, ctas // 2, slow_turn, 10_000_000, 200_000)
    assert [v for r, v in enumerate(got) if r != ctas // 2] == [-1.0] * (ctas - 1)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 7
    kda.check()
    assert exchange(ctas, 3) == summed(ctas, 3)
    x, g, do, h0, dht = make(1, 3000, 40, BF16, 7, 1)
    run(x, g, do, h0, dht)


@pytest.mark.parametrize("cu", [None, [0, 90, 200, 400]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinities(dtype, cu):
    """A state that meets an infinity is not finite from there to its sequence's end, as an infinity or a NaN,
    and nothing else is touched; the same for what comes back from an infinite gradient."""
    T, C = 400, 72
    x, g, do, h0, dht = make(1, T, C, dtype, 2, 1 if cu is None else len(cu) - 1)
    x[0, 100, 5], x[0, 127, 6], do[0, 150, 7], h0[0, 8] = float("inf"), -float("inf"), float("inf"), float("inf")
    dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, ht, saved = kda.gated_scan_fwd(x, g, h0, True, cu_seqlens=dev, save_for_backward=True)
    gr = kda.gated_scan_bwd(x, g, do, saved, dht=dht, initial_state=h0, cu_seqlens=dev)
    kda.check()
    first, last = (0, T) if cu is None else (90, 200)
    want = torch.zeros(T, C, dtype=torch.bool)
    want[100:last, 5] = want[127:last, 6] = True
    want[:T if cu is None else 90, 8] = True
    assert torch.equal(~torch.isfinite(o[0]).cpu(), want)
    assert torch.isinf(o[0, 100, 5]) and torch.isinf(o[0, 127, 6])
    want = torch.zeros(T, C, dtype=torch.bool)
    want[first:151, 7] = True
    assert torch.equal(~torch.isfinite(gr["dx"][0]).cpu(), want)
    dg = ~torch.isfinite(gr["dg"][0]).cpu()
    assert not dg[:, [c for c in range(C) if c not in (5, 6, 7, 8)]].any()
    h = torch.zeros(1, C, device="cuda")
    h[0, 3] = float("inf")
    step = kda.gated_scan_step(x[:, 0], g[:, 0], h)
    assert (~torch.isfinite(step)).nonzero().tolist() == [[0, 3]] == (~torch.isfinite(h)).nonzero().tolist()
