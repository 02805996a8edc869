"""The gated norm, the residual sum with its norm, and activations in 8 bits on the GPU, against
64-bit references; and a layer's operators together."""
import pytest
import torch

import gated_delta_rule_41_gb300 as kda
from block_util import (BF16, F32, check, d64, ref_add, ref_add_bwd, ref_gated, ref_pack, ref_scan,
                        ref_unpack)

pytestmark = pytest.mark.gpu
EPS = 1e-5
WIDTHS = [1, 2, 7, 8, 16, 31, 32, 33, 40, 64, 77, 96, 100, 128, 129, 200, 256, 257, 320, 512, 520, 1000, 1001,
          1024, 1032, 2048, 2056, 4096, 5120, 8192, 10000, 16383, 16384]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_41_gb300 import build
    build.build()


def rnd(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def sliced(t):
    """The same values as a slice of a wider tensor, whose tokens lie apart."""
    T, n = t.shape[0], t[0].numel() if t.shape[0] else 1
    wide = torch.full((T, 2 * n + 24), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, n + 8:2 * n + 8] = t.view(T, n)
    return wide[:, n + 8:2 * n + 8].view(t.shape)


def check_gated(x, z, w, act, dy, eps=EPS):
    y, x8, z8 = kda.gated_norm_fwd(x, z, w, eps=eps, act=act, keep8=True)
    ref = ref_gated(x, z, w, eps, act, dy)
    check("y", y, ref["y"], ref["y~"])
    assert torch.equal(y, kda.gated_norm_fwd(x, z, w, eps=eps, act=act))
    got = kda.gated_norm_bwd(x, z, w, dy, eps=eps, act=act)
    for n in ("dx", "dgate", "dw"):
        if got[n] is not None:
            check(n, got[n], ref[n], ref[n + "~"])
    # from 8 bits: what pack8 leaves, and the gradients at the values that it stands for
    for t, p in ((x, x8), (z, z8)):
        q = kda.pack8(t.contiguous())
        assert torch.equal(p.codes.view(torch.uint8), q.codes.view(torch.uint8))
        assert torch.equal(p.scales, q.scales)
    ref = ref_gated(kda.unpack8(x8, F32), kda.unpack8(z8, F32), w, eps, act, dy)
    got = kda.gated_norm_bwd(x8, z8, w, dy, eps=eps, act=act)
    for n in ("dx", "dgate", "dw"):
        if got[n] is not None:
            check(n + " of 8 bits", got[n], ref[n], ref[n + "~"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", WIDTHS)
def test_gated_widths(D, dtype):
    T, H = (3, 2) if D > 512 else (9, 3)
    x, z, dy = (rnd(D + i, T, H, D, dtype=dtype) for i in range(3))
    check_gated(x, z, 1 + 0.2 * rnd(5, D), "sigmoid" if D % 2 else "silu", dy)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,D", [(1, 1, 128), (1, 16, 128), (700, 5, 64), (333, 16, 128), (2000, 1, 256),
                                   (400, 3, 77), (5, 4000, 32)])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_rows(T, H, D, dtype, act):
    """Slices of wider projections; the weight in the tensors' type; no weight."""
    x, z, dy = (rnd(i, T, H, D, dtype=dtype) for i in range(3))
    w = (1 + 0.2 * rnd(5, D)).to(dtype)
    check_gated(sliced(x), sliced(4 * z), w, act, dy)
    check_gated(x, z, None, act, dy)


def test_gated_values():
    """Rows of zeros, gates far out on both sides, sizes far from one."""
    x, z, dy = (rnd(i, 12, 2, 64) for i in range(3))
    x[0], z[1], z[2] = 0.0, 60.0, -60.0
    x[3], x[4], dy[5] = x[3] * 1e15, x[4] * 1e-15, 0.0
    z[6], z[7] = 1e4, -1e4
    for act in ("sigmoid", "silu"):
        for t in (F32, BF16):
            check_gated(x.to(t), z.to(t), 1 + 0.2 * rnd(5, 64), act, dy.to(t))
    y = kda.gated_norm_fwd(x, z, None)
    assert (y[0] == 0).all() and torch.isfinite(y).all()


def test_gated_nan_stays_in_its_row():
    x, z, dy = (rnd(i, 9, 4, 128, dtype=BF16) for i in range(3))
    x[3, 1, 5], z[5, 2, 7] = float("nan"), float("inf")
    y, x8, z8 = kda.gated_norm_fwd(x, z, None, keep8=True)
    bad = torch.isnan(y)
    assert bad[3, 1].all() and not torch.isnan(kda.gated_norm_fwd(x, z, None)[5, 2, 7])
    bad[3, 1] = False
    assert not bad.any()
    assert torch.isnan(kda.unpack8(x8)[3, 1, 5]) and torch.isnan(kda.unpack8(z8)[5, 2, 7])


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("D", WIDTHS)
def test_add_widths(D, types):
    R, t = types
    T = 3 if D > 512 else 9
    r, x, dy, dr = rnd(D, T, D, dtype=R), rnd(1, T, D, dtype=t), rnd(2, T, D, dtype=t), rnd(3, T, D, dtype=R)
    run_add(r, x, 1 + 0.2 * rnd(5, D), 0.5 + 0.2 * rnd(6, D), dy, dr)


def run_add(r, x, w, alpha, dy, dr, eps=EPS):
    out, y = kda.add_norm_fwd(r, x, w, alpha=alpha, eps=eps)
    ref = ref_add(r, x, alpha, w, eps)
    check("r", out, ref["r"], ref["r~"])
    check("y", y, ref["y"], ref["y~"])
    got = kda.add_norm_bwd(out, w, dy, dr, x=x, alpha=alpha, eps=eps)
    ref = ref_add_bwd(out, w, dy, dr, x, alpha, eps)
    for n in ("dres", "dx", "dw", "dalpha"):
        if got[n] is not None:
            check(n, got[n], ref[n], ref[n + "~"])
    return got


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,D", [(1, 2048), (1500, 256), (700, 1000), (700, 1001), (4000, 40)])
@pytest.mark.parametrize("alpha", [None, 0.37, "vector"])
def test_add_rows(T, D, types, alpha):
    R, t = types
    r, x, dy, dr = rnd(9, T, D, dtype=R), rnd(1, T, D, dtype=t), rnd(2, T, D, dtype=t), rnd(3, T, D, dtype=R)
    w = (1 + 0.2 * rnd(5, D)).to(t)
    a = (0.5 + 0.2 * rnd(6, D)).to(t) if alpha == "vector" else alpha
    got = run_add(sliced(r), sliced(x), w, a, dy, dr)
    assert (got["dx"] is got["dres"]) == (alpha is None and R == t)
    run_add(r, x, None, a, dy, None)
    # the norm alone
    same, y = kda.add_norm_fwd(r, None, w)
    assert same is r
    ref = ref_add(r, None, None, w, EPS)
    check("y", y, ref["y"], ref["y~"])
    got = kda.add_norm_bwd(r, w, dy, None)
    ref = ref_add_bwd(r, w, dy, None, None, None, EPS)
    check("dres", got["dres"], ref["dres"], ref["dres~"])


def test_add_in_place():
    r, x = rnd(1, 50, 512, dtype=BF16), rnd(2, 50, 512, dtype=BF16)
    want, y = kda.add_norm_fwd(r, x, None, alpha=0.5)
    got, y2 = kda.add_norm_fwd(r, x, None, alpha=0.5, out_residual=r)
    assert got is r and torch.equal(want, r) and torch.equal(y, y2)
    dy, dr = rnd(3, 50, 512, dtype=BF16), rnd(4, 50, 512, dtype=BF16)
    a = kda.add_norm_bwd(r, None, dy, dr, alpha=0.5)
    b = kda.add_norm_bwd(r, None, dy, dr, alpha=0.5,
                         grads=dict(dres=dr, dx=torch.empty_like(dr)))
    assert torch.equal(a["dres"], dr) and torch.equal(a["dx"], b["dx"])


def test_empty_and_offsets():
    z = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    w = rnd(1, 64)
    assert kda.gated_norm_fwd(z, z, w).shape == z.shape
    got = kda.gated_norm_bwd(z, z, w, z)
    assert got["dx"].shape == z.shape and (got["dw"] == 0).all()
    z = torch.empty(0, 64, dtype=BF16, device="cuda")
    r, y = kda.add_norm_fwd(z, z, w, alpha=w)
    got = kda.add_norm_bwd(z, w, z, z, x=z, alpha=w)
    assert y.shape == z.shape and (got["dw"] == 0).all() and (got["dalpha"] == 0).all()
    p = kda.pack8(z)
    assert kda.unpack8(p).shape == z.shape
    # rows beyond 2^31 elements from the start
    far = 3 << 29
    big = torch.empty(2 * far + 256, dtype=BF16, device="cuda")
    x = big.as_strided((3, 2, 128), (far, 128, 1))
    v = rnd(2, 3, 2, 128, dtype=BF16)
    x.copy_(v)
    assert torch.equal(kda.gated_norm_fwd(x, v, None), kda.gated_norm_fwd(v, v, None))
    x2, v2 = x.view(3, 256), v.view(3, 256)
    a, b = kda.add_norm_fwd(x2, v2), kda.add_norm_fwd(v2, v2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(kda.pack8(x2).codes.view(torch.uint8), kda.pack8(v2).codes.view(torch.uint8))


def test_misaligned_pointers():
    """Tensors that start off a 16-byte boundary."""
    def off(t):
        flat = torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")
        flat[3:] = t.flatten()
        return flat[3:].view(t.shape)

    x, z, dy = (rnd(i, 40, 3, 128, dtype=BF16) for i in range(3))
    check_gated(off(x), off(z), off(1 + 0.2 * rnd(5, 128)), "silu", off(dy))
    r, x, dy, dr = (rnd(i, 40, 512, dtype=F32) for i in range(4))
    run_add(off(r), off(x), off(1 + rnd(5, 512)), off(rnd(6, 512)), off(dy), off(dr))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1,), (32,), (5, 31), (7, 32), (3, 33), (4, 5, 64), (9, 100), (2, 1111),
                                   (300, 128), (513, 2048), (1000, 40), (3, 7, 1), (4099, 77)])
def test_pack(shape, dtype):
    """Equal to the definition bit for bit, blocks of very unequal size among them."""
    x = rnd(sum(shape), *shape) * torch.exp(6 * rnd(1, *shape[:-1], 1))
    x = x.to(dtype)
    p = kda.pack8(x)
    codes, scales = ref_pack(x)
    assert torch.equal(p.scales.cpu(), scales)
    assert torch.equal(p.codes.cpu().double(), codes)
    want = ref_unpack(p.codes, p.scales)
    for t in (BF16, F32):
        assert torch.equal(d64(kda.unpack8(p, t)), want)
    big = (want - d64(x)).abs() / d64(x).abs().clamp(min=1e-300)
    scale = torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)[..., :shape[-1]]
    assert ((big <= 2.0 ** -4) | ((want - d64(x)).abs() <= scale * 2.0 ** -10)).all()


def test_pack_values():
    """Borders of the exponent, halves between codes, the largest and smallest numbers, zeros, and
    what is not finite."""
    x = torch.zeros(12, 32)
    x[1, 0], x[1, 1] = 448.0, 1.0
    x[2, 0], x[2, 1] = 448.0 * (1 + 2.0 ** -23), 1.0
    x[3, 0], x[3, 1] = 3.4028234663852886e38, -1.0
    x[4, :] = 2.0 ** -149
    x[5, 0], x[5, 1] = 2.0 ** -126, -2.0 ** -140
    x[6] = torch.arange(32) * 0.5 + 16.25            # halves between codes near 16 and 32
    x[6, 0] = 448.0
    x[7] = -x[6]
    x[8, 0], x[8, 1], x[8, 2], x[8, 3] = float("nan"), float("inf"), -float("inf"), 3.0
    x[9] = float("inf")
    x[10] = torch.arange(32) * 2.0 ** -11            # codes below the normal ones
    x[10, 0] = 256.0
    x[11, 3] = -0.0
    x = x.cuda()
    for t in (F32, BF16):
        for v in (x.to(t), x.to(t)[:, :31].contiguous(), x.to(t)[:, 3:]):
            p = kda.pack8(v)
            codes, scales = ref_pack(v)
            assert torch.equal(p.scales.cpu(), scales)
            got = p.codes.cpu().double()
            assert torch.equal(torch.isnan(got), torch.isnan(codes))
            assert torch.equal(got.nan_to_num(7.0), codes.nan_to_num(7.0))
            assert torch.equal(d64(kda.unpack8(p, F32)).nan_to_num(7.0),
                               ref_unpack(p.codes, p.scales).nan_to_num(7.0))


def test_pack_slices():
    """Rows that lie apart, with and without blocks that end inside the contiguous part."""
    wide = rnd(1, 6, 5, 400, dtype=BF16)
    whole = rnd(2, 6, 5, 384, dtype=BF16)        # blocks do not cross its rows: two of them are one
    for v in (wide[..., 8:136], wide[..., 3:100], wide[:, :, :32], whole[:, 1:3], wide[..., :1]):
        p, q = kda.pack8(v), kda.pack8(v.contiguous())
        assert p.shape == v.shape
        assert torch.equal(p.codes.view(torch.uint8), q.codes.view(torch.uint8))
        assert torch.equal(p.scales, q.scales)
    with pytest.raises(kda.KdaError):
        kda.pack8(wide.transpose(1, 2))
    with pytest.raises(kda.KdaError):
        kda.pack8(wide[:, 1:3])                  # 400 elements: the blocks of a row end with it
    with pytest.raises(kda.KdaError):
        kda.pack8(wide.half())


def test_chunk_scan_from_8_bits():
    """The chunk scan's backward takes kept inputs: its gradients are those at their values."""
    q, k, v, do = (rnd(i, 2, 128, 2, 64, dtype=BF16) for i in range(4))
    g = -rnd(5, 2, 128, 2, 64, dtype=BF16).abs()
    beta = torch.sigmoid(rnd(6, 2, 128, 2)).to(BF16)
    q8, k8, v8 = (kda.pack8(t) for t in (q, k, v))
    a = kda.chunk_kda_bwd(q8, k8, v8, g, beta, do, use_qk_l2norm_in_kernel=True)
    b = kda.chunk_kda_bwd(*(kda.unpack8(t) for t in (q8, k8, v8)), g, beta, do, use_qk_l2norm_in_kernel=True)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(a[n], b[n]), n
    cu = torch.tensor([0, 30, 128], dtype=torch.int32, device="cuda")
    one = [t[:1].contiguous() for t in (q, k, v, g, beta, do)]
    p = [kda.pack8(t) for t in one[:3]]
    a = kda.chunk_kda_bwd_varlen(*p, *one[3:5], one[5], cu, use_qk_l2norm_in_kernel=True)
    b = kda.chunk_kda_bwd_varlen(*(kda.unpack8(t) for t in p), *one[3:5], one[5], cu, use_qk_l2norm_in_kernel=True)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(a[n], b[n]), n
    kda.check()


def test_same_bits_in_graphs_and_on_streams():
    x, z, dy = (rnd(i, 500, 4, 128, dtype=BF16) for i in range(3))
    r, u = rnd(7, 500, 512, dtype=F32), rnd(8, 500, 512, dtype=F32)
    w, w2, al = rnd(5, 128), rnd(6, 512), rnd(9, 512)

    def all_of(stream=None):
        y, x8, z8 = kda.gated_norm_fwd(x, z, w, keep8=True, stream=stream)
        out, n = kda.add_norm_fwd(r, y.view(500, 512), w2, alpha=al, stream=stream)
        a = kda.add_norm_bwd(out, w2, n, u, x=y.view(500, 512), alpha=al, stream=stream)
        b = kda.gated_norm_bwd(x8, z8, w, a["dx"].view(500, 4, 128), stream=stream)
        p = kda.unpack8(kda.pack8(out, stream=stream), F32, stream=stream)
        return [y, out, n, *a.values(), *b.values(), p]

    want = all_of()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    others, here = all_of(side), all_of()
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(want, others, here):
        assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for t in got:
        t.zero_()
    graph.replay()
    graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_refusals():
    x = rnd(1, 10, 2, 64, dtype=BF16)

    def refused(status, f, *a, **k):
        with pytest.raises(kda.KdaError) as e:
            f(*a, **k)
        assert e.value.status == status

    refused(1, kda.gated_norm_fwd, x, x.float())
    refused(3, kda.gated_norm_fwd, x.half(), x.half())
    refused(1, kda.gated_norm_fwd, x, x, act="tanh")
    refused(1, kda.gated_norm_fwd, x, x, eps=0.0)
    refused(1, kda.gated_norm_fwd, x, x, rnd(1, 63))
    refused(1, kda.gated_norm_fwd, x, x[:5])
    refused(1, kda.gated_norm_fwd, x.transpose(0, 1), x.transpose(0, 1))
    refused(1, kda.gated_norm_fwd, x, x.cpu())
    refused(3, kda.gated_norm_fwd, rnd(1, 1, 1, 16385), rnd(1, 1, 1, 16385))
    refused(1, kda.gated_norm_bwd, kda.pack8(x), x, None, x)
    refused(1, kda.gated_norm_bwd, x, x, None, x.float())
    r = x.view(10, 128)
    refused(1, kda.add_norm_fwd, r, r.float().cpu())
    refused(3, kda.add_norm_fwd, r, r.float())
    refused(1, kda.add_norm_fwd, r, r, eps=-1.0)
    refused(1, kda.add_norm_fwd, r, r, alpha=float("nan"))
    refused(1, kda.add_norm_fwd, r, r[:, :64])
    refused(1, kda.add_norm_fwd, r, r, rnd(1, 128), alpha=rnd(1, 128, dtype=BF16))
    refused(1, kda.add_norm_bwd, r, None, r, alpha=rnd(1, 128))
    refused(2, kda.add_norm_fwd, r[:1].expand(10, 128), r)
    refused(1, kda.Packed8, r, r)
    with pytest.raises(kda.KdaError):
        kda.unpack8(kda.pack8(r), torch.float16)


@pytest.mark.parametrize("cu", [None, [0, 40, 40, 96]])
def test_a_layer(cu):
    """Recurrence, gated norm (its inputs kept in 8 bits), projection, residual sum and norm, forward
    and backward as a training step calls them, against the same formulas in 64 bits."""
    T, H, D = 96, 2, 64
    C = H * D
    x, g, z = rnd(1, 1, T, C), -rnd(2, 1, T, C).abs() * 0.2, rnd(3, T, H, D)
    res, up, dy = rnd(4, T, C), rnd(5, T, C), rnd(6, T, C)
    w, w2, al, proj = 1 + 0.1 * rnd(7, D), 1 + 0.1 * rnd(8, C), 0.5 + 0.1 * rnd(9, C), rnd(10, C, C) / C ** 0.5
    dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, _, saved = kda.gated_scan_fwd(x, g, tied=True, cu_seqlens=dev, save_for_backward=True)
    y, o8, z8 = kda.gated_norm_fwd(o.view(T, H, D), z, w, keep8=True)
    b = y.view(T, C) @ proj
    r, n = kda.add_norm_fwd(res, b, w2, alpha=al)
    ga = kda.add_norm_bwd(r, w2, dy, up, x=b, alpha=al)
    gg = kda.gated_norm_bwd(o8, z8, w, (ga["dx"] @ proj.T).view(T, H, D))
    gs = kda.gated_scan_bwd(x, g, gg["dx"].view(1, T, C), saved, tied=True, cu_seqlens=dev)
    kda.check()
    scan = ref_scan(x, g, None, True, cu)
    gated = ref_gated(scan["o"].view(T, H, D), z, w, EPS, "sigmoid")
    rb = gated["y"].view(T, C) @ d64(proj)
    add = ref_add(res, rb, al, w2, EPS)
    ra = ref_add_bwd(add["r"], w2, dy, up, rb, al, EPS)
    rg = ref_gated(kda.unpack8(o8, F32), kda.unpack8(z8, F32), w, EPS, "sigmoid",
                   (ra["dx"] @ d64(proj).T).view(T, H, D))
    rs = ref_scan(x, g, None, True, cu, rg["dx"].view(1, T, C))
    # each value passes a few 32-bit operators, a product of 128 terms among them: 2^-14 of its kind's
    # size is far beyond their roundings
    for name, got, want in (("o", o, scan["o"]), ("y", y, gated["y"]), ("r", r, add["r"]), ("n", n, add["y"]),
                            ("dres", ga["dres"], ra["dres"]), ("dalpha", ga["dalpha"], ra["dalpha"]),
                            ("dw2", ga["dw"], ra["dw"]), ("do", gg["dx"], rg["dx"]), ("dz", gg["dgate"], rg["dgate"]),
                            ("dw", gg["dw"], rg["dw"]), ("dx", gs["dx"], rs["dx"]), ("dg", gs["dg"], rs["dg"])):
        err = (d64(got).view(want.shape) - want).norm() / want.norm()
        assert err < 2.0 ** -14, (name, float(err))


@pytest.mark.parametrize("less", [31, 1])
def test_pack_of_the_longest_rows(less):
    """A row of 2^31 - 31 and of 2^31 - 1 elements: its last blocks, and some in between."""
    D = (1 << 31) - less
    x = torch.zeros(1, D, dtype=BF16, device="cuda")
    places = [0, 1 << 20, (1 << 30) - 32, (1 << 31) - 4096 - 64, (D - 1) // 32 * 32 - 64]
    parts = [slice(p, min(p + 160, D)) for p in places]
    for i, s in enumerate(parts):
        x[0, s] = rnd(i, x[0, s].shape[0], dtype=BF16)
    p = kda.pack8(x)
    for s in parts:
        codes, scales = ref_pack(x[:, s])
        assert torch.equal(p.codes[:, s].cpu().double(), codes)
        assert torch.equal(p.scales[:, s.start // 32:-(-s.stop // 32)].cpu(), scales)
    back = kda.unpack8(p)
    for s in parts:
        b = slice(s.start // 32, -(-s.stop // 32))
        assert torch.equal(d64(back[:, s]), ref_unpack(p.codes[:, s], p.scales[:, b]))
    assert int(torch.count_nonzero(back.view(torch.int16))) <= 160 * len(parts)


# Rows by which a CTA's groups of threads come to their ring's slots again: each shape has more than twice
# as many turns as the ring has slots (four, three or two; two or three CTAs of an SM, seven for the
# smallest rings), and a last turn that some groups do not have.
RINGS = [(BF16, BF16, 9583, 2048), (BF16, BF16, 16421, 1024), (BF16, BF16, 4111, 4096), (BF16, BF16, 2135, 8192),
         (BF16, BF16, 767, 16384), (F32, F32, 9583, 1024), (F32, F32, 2135, 4096), (F32, BF16, 9583, 1024),
         (F32, BF16, 1527, 8192), (BF16, BF16, 25003, 77)]


@pytest.mark.parametrize("R,t,T,D", RINGS)
def test_add_many_turns(R, t, T, D):
    r, x, dy, dr = rnd(9, T, D, dtype=R), rnd(1, T, D, dtype=t), rnd(2, T, D, dtype=t), rnd(3, T, D, dtype=R)
    run_add(r, sliced(x), 1 + 0.2 * rnd(5, D), 0.5 + 0.2 * rnd(6, D), dy, dr)


GATED_RINGS = [(BF16, 10303, 5, 128), (BF16, 643, 5, 2048), (BF16, 1851, 5, 1024), (F32, 4801, 5, 128),
               (F32, 1851, 5, 512), (BF16, 2003, 5, 77)]


@pytest.mark.parametrize("dtype,T,H,D", GATED_RINGS)
def test_gated_many_turns(dtype, T, H, D):
    """Five heads: a step over rows carries from the head into the token."""
    x, z, dy = (rnd(i, T, H, D, dtype=dtype) for i in range(3))
    check_gated(sliced(x), sliced(z), 1 + 0.2 * rnd(5, D), "silu", dy)


def counted(name, got, one, rows):
    """Sums of ``rows`` equal terms, none left out and none taken twice.  A sum passes at most 22 rows of a
    thread, 32 groups of a CTA, 38 partial rows of a warp and 5 steps among the warps, each rounded once, as
    is the one term: 98 * 2^-24 of it, under a third of one of 51,515 terms."""
    want = d64(one) * rows
    assert ((d64(got) - want).abs() <= 98 * 2.0 ** -24 * want.abs()).all(), name


@pytest.mark.parametrize("R,t,T,D", RINGS)
def test_add_counts_every_row(R, t, T, D):
    def rows(n, *a, **k):
        return rnd(*a, 1, D, **k).expand(n, D).contiguous()

    w, al = 1 + 0.2 * rnd(5, D), 0.5 + 0.2 * rnd(6, D)
    got, one = (kda.add_norm_bwd(rows(n, 1, dtype=R), w, rows(n, 2, dtype=t), rows(n, 3, dtype=R),
                                 x=rows(n, 4, dtype=t), alpha=al) for n in (T, 1))
    for n in ("dw", "dalpha"):
        counted(n, got[n], one[n], T)
    for n in ("dres", "dx"):
        assert torch.equal(got[n], one[n].expand(T, D)), n


@pytest.mark.parametrize("dtype,T,H,D", GATED_RINGS)
def test_gated_counts_every_row(dtype, T, H, D):
    def rows(n, seed):
        return rnd(seed, 1, 1, D, dtype=dtype).expand(n, H, D).contiguous()

    w = 1 + 0.2 * rnd(5, D)
    for packed in (False, True):
        got, one = (kda.gated_norm_bwd(*((kda.pack8(t) if packed else t) for t in (rows(n, 1), rows(n, 2))), w,
                                       rows(n, 3)) for n in (T, 1))
        alone = kda.gated_norm_bwd(*((kda.pack8(t) if packed else t) for t in (rows(1, 1)[:, :1], rows(1, 2)[:, :1])),
                                   w, rows(1, 3)[:, :1].contiguous())
        counted("dw", got["dw"], alone["dw"], T * H)
        for n in ("dx", "dgate"):
            assert torch.equal(got[n], one[n].expand(T, H, D)), n


def test_unpack_to_bf16_rounds_what_it_cannot_hold():
    """Codes of blocks at the least scale reach 2^-135: exact in float32, in bf16 rounded to its smallest
    steps of 2^-133, halves to even."""
    x = torch.arange(-64, 64).float().view(4, 32) * 2.0 ** -135
    x[1, 0] = 2.0 ** -120
    for D in (32, 31):
        p = kda.pack8(x[:, :D].contiguous().cuda())
        assert (p.scales == 1).all()
        want = ref_unpack(p.codes, p.scales)
        assert torch.equal(d64(kda.unpack8(p, F32)), want)
        got = kda.unpack8(p, BF16)
        assert torch.equal(d64(got), (want * 2.0 ** 133).round() * 2.0 ** -133)
        assert not torch.equal(d64(got), want)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 33), (F32, 64)])
def test_gates_far_out(dtype, D, act):
    """Gates past |z| = 87, whose sigmoid or its derivative is among the subnormal numbers (of float32 down
    to z = -104, of bf16 to -93), and on to where nothing is left.  A rounding there is off by half of
    2^-149; a result passes a handful of products of such numbers with others that are under 100 here."""
    z = torch.linspace(-112, 112, 113 * D).view(113, 1, D).to(dtype).cuda()
    x, dy = rnd(1, 113, 1, D, dtype=dtype), rnd(2, 113, 1, D, dtype=dtype)
    w = 1 + 0.2 * rnd(5, D)
    tiny = 8 * 100 * 2.0 ** -150
    y, x8, z8 = kda.gated_norm_fwd(x, z, w, act=act, keep8=True)
    ref = ref_gated(x, z, w, EPS, act, dy)
    check("y", y, ref["y"], ref["y~"] + tiny)
    if dtype == F32:
        assert (y[9:20] != 0).all()               # z from -94 to -72: none is lost
    got = kda.gated_norm_bwd(x, z, w, dy, act=act)
    of8 = kda.gated_norm_bwd(x8, z8, w, dy, act=act)
    ref8 = ref_gated(kda.unpack8(x8, F32), kda.unpack8(z8, F32), w, EPS, act, dy)
    for n in ("dx", "dgate"):
        check(n, got[n], ref[n], ref[n + "~"] + tiny)
        check(n + " of 8 bits", of8[n], ref8[n], ref8[n + "~"] + tiny)


@pytest.mark.parametrize("eps", [1e-5, 1e-30, 1e-40])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_zeros(dtype, eps):
    """A row of zeros has the gradients that its epsilon makes, of whatever size that is."""
    r, dy, dr, z = (rnd(i, 3, 64, dtype=dtype) for i in range(4))
    r[1], w = 0.0, 1 + 0.2 * rnd(5, 64)
    got, ref = kda.add_norm_bwd(r, w, dy, dr, eps=eps), ref_add_bwd(r, w, dy, dr, None, None, eps)
    for n in ("dres", "dw"):
        check(n, got[n], ref[n], ref[n + "~"])
    x, z, up = (t.view(3, 1, 64) for t in (r, z, dy))
    got, ref = kda.gated_norm_bwd(x, z, w, up, eps=eps), ref_gated(x, z, w, eps, "sigmoid", up)
    for n in ("dx", "dgate", "dw"):
        check(n, got[n], ref[n], ref[n + "~"])
