"""64-bit references of the operators around a mixing layer, on the CPU, and bounds for what the
kernels' 32-bit arithmetic and one rounding of each result may be off by."""
import torch

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}     # a rounding: half a step, relative


def d64(t):
    return None if t is None else t.detach().cpu().double()


def seqs_of(x, cu):
    """(batch entry, first, end, row of the states) of every sequence."""
    if cu is None:
        return [(b, 0, x.shape[1], b) for b in range(x.shape[0])]
    return [(0, a, b, i) for i, (a, b) in enumerate(zip(cu, cu[1:]))]


def _line(a, u, h):
    out = torch.empty_like(u)
    for t in range(u.shape[0]):
        h = a[t] * h + u[t]
        out[t] = h
    return out, h


def ref_scan(x, g, h0=None, tied=False, cu=None, do=None, dht=None):
    """dict of o, ht (and dx, dg, dh0), each with a bound under "name~".

    The bound of a state: a step rounds twice, 2^-23 of the magnitudes that meet in it, and its
    decay is off by 2^-22 of 1 - exp(g) (or of exp(g), where that is small); these errors decay as
    states do.  Runs of tokens are combined with one more product.  With H the same recurrence
    on magnitudes, the error is under 2^-21 E, E the recurrence with H as its input.

    What a strong decay leaves, m = exp(g) l, is off by more of itself: the exponential's argument
    g log2(e) carries two roundings, 2^-23 |g| of the result; and a decay under 2^-126 counts as that."""
    x, g, h0, do, dht = (d64(t) for t in (x, g, h0, do, dht))
    a, c = g.exp(), -torch.expm1(g) if tied else torch.ones_like(g)
    C = x.shape[2]
    rows = x.shape[0] if cu is None else len(cu) - 1
    zero = torch.zeros(rows, C, dtype=torch.float64)
    h0, dht = zero if h0 is None else h0, zero if dht is None else dht
    r = {n: torch.empty_like(x) for n in ("o", "o~", "dx", "dx~", "dg", "dg~")}
    r.update({n: zero.clone() for n in ("ht", "ht~", "dh0", "dh0~")})
    u = 2.0 ** -21
    for b, lo, hi, s in seqs_of(x, cu):
        A, U, X = a[b, lo:hi], (c * x)[b, lo:hi], x[b, lo:hi]
        o, end = _line(A, U, h0[s])
        H, _ = _line(A, U.abs(), h0[s].abs())
        E, _ = _line(A, H, torch.zeros(C, dtype=torch.float64))
        r["o"][b, lo:hi], r["o~"][b, lo:hi] = o, u * E
        r["ht"][s], r["ht~"][s] = end, u * E[-1] if hi > lo else 0
        if do is None:
            continue
        D = do[b, lo:hi]
        shift = lambda v, first: torch.cat([first[None], v[:-1]])  # noqa: E731
        # m_t = a_t (do_t + m_{t+1}): the recurrence from the other end
        back = lambda v, m: tuple(t.flip(0) if t.dim() == 2 else t  # noqa: E731
                                  for t in _line(A.flip(0), (A * v).flip(0), m))
        m, m1 = back(D, dht[s])
        M, _ = back(D.abs(), dht[s].abs())
        EM, _ = _line(A.flip(0), M.flip(0), torch.zeros(C, dtype=torch.float64))
        EM = EM.flip(0)
        far = D.abs() + torch.cat([M[1:], dht[s].abs()[None]])
        # (what the least decay makes is itself rounded, three times)
        far = far * (2.0 ** -23 * torch.nan_to_num(A * g[b, lo:hi].abs()) + 2.0 ** -126 * (1 + 2.0 ** -20)) / u
        EM = EM + far
        up = lambda v, last: torch.cat([v[1:], last[None]])  # noqa: E731
        lam = D + up(m, dht[s])
        LAM, EL = D.abs() + up(M, dht[s].abs()), up(EM, torch.zeros(C, dtype=torch.float64))
        cc = c[b, lo:hi]
        r["dx"][b, lo:hi] = cc * lam
        r["dx~"][b, lo:hi] = u * cc * (EL + LAM)
        w = shift(o, h0[s]) - (X if tied else 0)
        W = shift(H, h0[s].abs()) + (X.abs() if tied else 0)
        EW = shift(E, torch.zeros(C, dtype=torch.float64))
        r["dg"][b, lo:hi] = m * w
        # a product's error: each factor's error times the other, and the two errors; an m among the
        # subnormal numbers is a multiple of 2^-149
        r["dg~"][b, lo:hi] = u * (EM * W + M * (EW + W)) + u * u * EM * EW + 2.0 ** -149 * W
        r["dh0"][s], r["dh0~"][s] = m1, u * EM[0] if hi > lo else 0
    return r


def check(name, got, ref, slack, dtype=None):
    """|got - ref| is at most half a step of its type beyond slack; equal where not finite."""
    t = got.dtype if dtype is None else dtype
    got = d64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN elsewhere"
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), name
    slack = torch.as_tensor(slack, dtype=torch.float64).expand(ref.shape)
    # the type's smallest steps round to multiples of 2^-133 (bf16) or 2^-149
    bound = HALF[t] * (ref.abs() + slack) + slack + (2.0 ** -133 if t == BF16 else 2.0 ** -149)
    over = (got - ref).abs() - bound
    over = over[fine]
    if over.numel() and over.max() > 0:
        worst = ((got - ref).abs() / bound)[fine].max()
        raise AssertionError(f"{name}: {int((over > 0).sum())} of {over.numel()} off, worst "
                             f"{worst:.3g} of its bound")


def _gates(z, act):
    # 1 - sigmoid(z) as sigmoid(-z): the difference has no digits left at z = 60, in 64 bits too
    s, other = torch.sigmoid(z), torch.sigmoid(-z)
    return (s, s * other) if act == "sigmoid" else (z * s, s * (1 + z * other))


def ref_gated(x, z, w, eps, act, dy=None):
    """dict y (dx, dgate, dw), each with its bound under "name~".

    Sums over a row are 32-bit, at most 64 additions deep: 2^-18 of the magnitudes; an
    exponential's argument is rounded, 2^-23 |z| of the gate; the rest is a dozen roundings."""
    x, z, w, dy = (d64(t) for t in (x, z, w, dy))
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    s, ds = _gates(z, act)
    n, u = x * r, 2.0 ** -18 + 2.0 ** -22 * z.abs()
    # the gate's derivative is a product of two factors, for silu a sum with cancellation
    ads = ds.abs() if act == "sigmoid" else torch.sigmoid(z) * (1 + z.abs() * torch.sigmoid(-z))
    out = {"y": n * w * s}
    out["y~"] = u * out["y"].abs()
    if dy is None:
        return out
    dn = dy * w * s
    out["dx"] = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    mean = (u * (dn * n).abs()).mean(-1, keepdim=True)
    out["dx~"] = r * (u * dn.abs() + n.abs() * (mean + 2.0 ** -18 * (dn * n).abs().mean(-1, keepdim=True)))
    out["dgate"] = dy * n * w * ds
    out["dgate~"] = 2 * u * (dy * n * w).abs() * ads
    flat = (dy * n * s).flatten(0, -2)
    out["dw"] = flat.sum(0)
    # rows are added up one after the other: 2^-24 of the magnitudes for each
    out["dw~"] = ((u.flatten(0, -2) + 2.0 ** -24 * flat.shape[0]) * flat.abs()).sum(0)
    return out


def ref_add(r, x, alpha, w, eps):
    r, x, w = d64(r), d64(x), d64(w)
    alpha = 1.0 if alpha is None else d64(alpha) if isinstance(alpha, torch.Tensor) else alpha
    s = r if x is None else r + alpha * x
    inv = 1 / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    mag = r.abs() + (0 if x is None else (alpha * x).abs())
    w = torch.ones(r.shape[-1], dtype=torch.float64) if w is None else w
    out = {"r": s, "r~": 2.0 ** -23 * mag, "y": w * s * inv}
    out["y~"] = 2.0 ** -18 * (w * mag * inv).abs()
    return out


def ref_add_bwd(r, w, dy, dres, x, alpha, eps):
    r, w, dy, dres, x = (d64(t) for t in (r, w, dy, dres, x))
    vec = isinstance(alpha, torch.Tensor)
    alpha = 1.0 if alpha is None else d64(alpha) if vec else alpha
    w = torch.ones(r.shape[-1], dtype=torch.float64) if w is None else w
    inv = 1 / (r.square().mean(-1, keepdim=True) + eps).sqrt()
    n, dn, u = r * inv, dy * w, 2.0 ** -18
    up = torch.zeros_like(r) if dres is None else dres
    out = {"dres": up + inv * (dn - n * (dn * n).mean(-1, keepdim=True))}
    slack = u * (up.abs() + inv * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True)))
    out["dres~"], out["dx"], out["dx~"] = slack, alpha * out["dres"], abs(alpha) * slack
    rows = u + 2.0 ** -24 * r.shape[0]
    out["dw"], out["dw~"] = (dy * n).sum(0), rows * (dy * n).abs().sum(0)
    if vec:
        out["dalpha"] = (out["dres"] * x).sum(0)
        out["dalpha~"] = (rows * (out["dres"] * x).abs() + (slack * x).abs()).sum(0)
    return out


def ref_pack(x):
    """(codes as values, scale bytes) with the exponent found by trying every one."""
    x = d64(x)
    n = x.shape[-1]
    fine = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    pad = torch.cat([fine, torch.zeros(*x.shape[:-1], -n % 32, dtype=torch.float64)], -1)
    top = pad.unflatten(-1, (-1, 32)).abs().amax(-1)
    e = torch.full(top.shape, -126, dtype=torch.int64)
    for k in range(-126, 121):
        e = torch.where(top > 448 * 2.0 ** k, torch.full_like(e, k + 1), e)
    scale = torch.pow(2.0, e.double()).repeat_interleave(32, -1)[..., :n]
    # |x / scale| <= 448 on a grid of 2^-9, or of 2^-3 of the leading bit
    v = fine / scale
    _, k = torch.frexp(v.abs().clamp(min=2.0 ** -6))
    step = torch.pow(2.0, (k - 4).double())
    code = (v / step).round() * step              # halves to even
    # 256 * 2^120 is no float32: the code below it
    code = torch.where((scale == 2.0 ** 120) & (code.abs() >= 256), code.sign() * 240, code)
    return torch.where(torch.isfinite(x), code, torch.full_like(code, float("nan"))), (e + 127).to(torch.uint8)


def ref_unpack(codes, scales):
    s = torch.pow(2.0, scales.cpu().double() - 127).repeat_interleave(32, -1)[..., :codes.shape[-1]]
    return codes.cpu().float().double() * s
