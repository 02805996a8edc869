"""Cases of the operators around a sequence-mixing layer: the gated linear recurrence over long
sequences, the gated norm after a mixing layer, the residual sum with the norm before the next one,
and activations kept in 8 bits for the backward pass.

Each case has a plain form in elementary torch operations (``own`` false), the framework's calls
(``own`` true) and a 64-bit evaluation of the operator's definition (``exact``).

Definitions, per channel, row and block:

    recurrence   h_t = exp(g_t) h_{t-1} + c_t x_t,  c_t = 1, or 1 - exp(g_t) when tied;  o_t = h_t
                 m_t = exp(g_t) l_t,  l_t = do_t + m_{t+1}  (m behind the last token: dht)
                 dx_t = c_t l_t,  dg_t = m_t (h_{t-1} - [tied] x_t),  dh0 = m_1
    gated norm   n = x / sqrt(mean(x^2) + eps),  y = n w s(z);  s = sigmoid or z sigmoid(z)
                 dn = dy w s(z),  dx = (dn - n mean(dn n)) / sqrt(mean(x^2) + eps),
                 dz = dy n w s'(z),  dw = sum over rows of dy n s(z)
    add norm     r' = r + alpha x,  y = w r' / sqrt(mean(r'^2) + eps)
                 dr = dr' + (dn - n mean(dn n)) / sqrt(...), dn = dy w;  dx = alpha dr,
                 dw = sum dy n,  dalpha = sum dr x
    8 bits       blocks of 32 neighbours share the smallest 2^e, e >= -126, with
                 max |x| <= 448 * 2^e; kept are the e4m3 codes of x / 2^e and e + 127
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-5
BLOCK = 32


# ---- the cases -----------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch of 256 sequences: latency
        dict(name="step_batch", op="step", B=256, C=2048, t="bf16", tied=True),
        # the training shape of a layer of 16 heads of 128
        dict(name="scan_train_fwd", op="scan", way="fwd", B=4, T=8192, C=2048, t="bf16", tied=False,
             seqs=0, salt=0, h0=False),
        dict(name="scan_train_bwd", op="scan", way="bwd", B=4, T=8192, C=2048, t="bf16", tied=False,
             seqs=0, salt=0, h0=False),
        # one long document through a narrow layer: few channels, a long axis
        dict(name="scan_long_fwd", op="scan", way="fwd", B=1, T=65536, C=512, t="f32", tied=True,
             seqs=0, salt=0, h0=True),
        # sequences of unequal length packed together, in training
        dict(name="scan_packed_bwd", op="scan", way="bwd", B=1, T=32768, C=1000, t="bf16", tied=True,
             seqs=16, salt=3, h0=True),
        # the heads of a few tokens that are being decoded: latency
        dict(name="gated_decode", op="gated", way="fwd", T=8, H=16, D=128, t="bf16", act="sigmoid",
             keep=False),
        # the training shape, inputs kept in 8 bits on the way
        dict(name="gated_train_fwd8", op="gated", way="fwd", T=32768, H=16, D=128, t="bf16",
             act="sigmoid", keep=True),
        # and the backward pass that reads them
        dict(name="gated_train_bwd8", op="gated", way="bwd", T=32768, H=16, D=128, t="bf16",
             act="sigmoid", keep=True),
        # between two blocks of the same model
        dict(name="add_train_fwd", op="add", way="fwd", T=32768, D=2048, t="bf16", res="bf16",
             alpha="vector"),
        # the same with a residual stream in 32 bits, an odd number of tokens
        dict(name="add_train_bwd", op="add", way="bwd", T=20011, D=2048, t="bf16", res="f32",
             alpha="vector"),
        # an activation of the training shape kept for the backward pass
        dict(name="pack_train", op="pack", way="fwd", T=32768, D=2048, t="bf16"),
        # and one of an odd width given back in 32 bits
        dict(name="unpack_odd", op="pack", way="bwd", T=4099, D=1111, t="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random())) if hi > lo else lo


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan", "gated", "gated", "add", "add", "pack"])
    t, way = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["fwd", "bwd"])
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 512), C=_log_int(rng, 50, 8192), t=t, tied=rng.random() < 0.5)
    if op == "scan":
        C, seqs = _log_int(rng, 60, 4096), rng.choice([0, 0, _log_int(rng, 1, 64)])
        if rng.random() < 0.6:
            C = max(64, C // 64 * 64)
        B = 1 if seqs else rng.choice([1, 1, 2, 3, 4])
        most = min(65536, (1 << 25) // (B * C))
        return dict(op=op, way=way, B=B, T=_log_int(rng, 30, most), C=C, t=t, tied=rng.random() < 0.5,
                    seqs=seqs, salt=rng.randrange(1000), h0=rng.random() < 0.5)
    if op == "gated":
        D, H = rng.choice([32, 64, 100, 128, 192, 256, 512, 2048, 77]), rng.choice([1, 2, 4, 5, 16])
        return dict(op=op, way=way, T=_log_int(rng, 1, (1 << 25) // (D * H)), H=H, D=D, t=t,
                    act=rng.choice(["sigmoid", "silu"]), keep=rng.random() < 0.5)
    D = rng.choice([512, 1000, 1024, 1536, 2048, 4096, 5120, 8192, 1001, 77])
    T = _log_int(rng, 1, (3 << 23) // D)
    if op == "pack":
        return dict(op=op, way=way, T=T, D=D, t=t)
    return dict(op=op, way=way, T=T, D=D, t=t, res="f32" if t == "f32" else rng.choice(["bf16", "f32"]),
                alpha=rng.choice(["none", "number", "vector"]))


def _lens(c):
    """Lengths of the packed sequences, spread by golden-ratio steps; they sum to T and may be 0."""
    w = [0.2 + (0.137 * c["salt"] + 0.6180339887498949 * (i + 1)) % 1.0 for i in range(c["seqs"])]
    cuts = [0]
    for x in w:
        cuts.append(cuts[-1] + x)
    cuts = [int(round(c["T"] * x / cuts[-1])) for x in cuts]
    return [b - a for a, b in zip(cuts, cuts[1:])]


# ---- inputs --------------------------------------------------------------------------------

def _log_decay(gen, *shape):
    """Log-decays of a trained layer: half-lives from under a token to some thousands of them."""
    return -torch.exp(1.5 * torch.randn(*shape, generator=gen, device=DEV) - 4.0)


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st, t = dict(c=c), TYPES[c["t"]]

    def randn(*shape, dtype=t):
        return torch.randn(*shape, generator=gen, device=DEV).to(dtype)

    if own:
        import gated_delta_rule_41_gb300 as kda
        st["kda"] = kda
    if c["op"] == "step":
        st["x"], st["g"] = randn(c["B"], c["C"]), _log_decay(gen, c["B"], c["C"]).to(t)
        st["h"] = randn(c["B"], c["C"], dtype=F32)
        st["next"] = torch.empty_like(st["h"])   # states of two steps, used in turn
    elif c["op"] == "scan":
        B, T, C, N = c["B"], c["T"], c["C"], c["seqs"] or c["B"]
        st["x"], st["g"] = randn(B, T, C), _log_decay(gen, B, T, C).to(t)
        st["h0"] = randn(N, C, dtype=F32) if c["h0"] else None
        cu = [0]
        for n in _lens(c) if c["seqs"] else [T] * B:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        if c["way"] == "bwd":
            st["do"], st["dht"] = randn(B, T, C), randn(N, C, dtype=F32) if c["h0"] else None
            if own:
                st["saved"] = kda.gated_scan_fwd(st["x"], st["g"], st["h0"], tied=c["tied"],
                                                 cu_seqlens=st["cu"] if c["seqs"] else None,
                                                 save_for_backward=True)[2]
    elif c["op"] == "gated":
        T, H, D = c["T"], c["H"], c["D"]
        st["x"], st["w"] = randn(T, H, D), 1.0 + 0.1 * randn(D, dtype=F32)
        # the gate is a slice of a wider projection's output
        st["z"] = randn(T, 2 * H * D)[:, H * D:].view(T, H, D)
        if c["way"] == "bwd":
            st["dy"] = randn(T, H, D)
            if c["keep"]:
                st["x8"], st["z8"] = _plain_pack(st["x"]), _plain_pack(st["z"])
                if own:
                    st["x8"], st["z8"] = kda.Packed8(*st["x8"]), kda.Packed8(*st["z8"])
    elif c["op"] == "add":
        T, D = c["T"], c["D"]
        st["r"], st["x"] = 2.0 * randn(T, D, dtype=TYPES[c["res"]]), randn(T, D)
        st["w"] = 1.0 + 0.1 * randn(D, dtype=F32)
        st["alpha"] = {"none": None, "number": 0.5, "vector": 0.5 + 0.1 * randn(D, dtype=F32)}[c["alpha"]]
        if c["way"] == "bwd":
            st["dy"], st["dr"] = randn(T, D), randn(T, D, dtype=TYPES[c["res"]])
    else:
        # activations differ in size from channel to channel
        st["x"] = (randn(c["T"], c["D"], dtype=F32) * torch.exp(randn(c["D"], dtype=F32))).to(t)
        if c["way"] == "bwd":
            st["code"], st["e"] = _plain_pack(st["x"])
            if own:
                st["x8"] = kda.Packed8(st["code"], st["e"])
    return st


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    st, c = state, state["c"]
    return _own(st, c, st["kda"]) if own else _plain(st, c)


def _own(st, c, kda):
    op, way = c["op"], c.get("way")
    if op == "step":
        o = kda.gated_scan_step(st["x"], st["g"], st["h"], tied=c["tied"], new_state=st["next"])
        return dict(o=o, h=st["next"])
    if op == "scan":
        cu = st["cu"] if c["seqs"] else None
        if way == "fwd":
            o, ht, _ = kda.gated_scan_fwd(st["x"], st["g"], st["h0"], output_final_state=True,
                                          tied=c["tied"], cu_seqlens=cu, save_for_backward=True)
            return dict(o=o, ht=ht)
        grads = kda.gated_scan_bwd(st["x"], st["g"], st["do"], st["saved"], dht=st["dht"],
                                   initial_state=st["h0"], tied=c["tied"], cu_seqlens=cu)
        return {k: v for k, v in grads.items() if v is not None}
    if op == "gated":
        if way == "fwd" and c["keep"]:
            y, x8, z8 = kda.gated_norm_fwd(st["x"], st["z"], st["w"], eps=EPS, act=c["act"], keep8=True)
            return dict(y=y, xc=x8.codes, xe=x8.scales, zc=z8.codes, ze=z8.scales)
        if way == "fwd":
            return dict(y=kda.gated_norm_fwd(st["x"], st["z"], st["w"], eps=EPS, act=c["act"]))
        x, z = (st["x8"], st["z8"]) if c["keep"] else (st["x"], st["z"])
        return kda.gated_norm_bwd(x, z, st["w"], st["dy"], eps=EPS, act=c["act"])
    if op == "add":
        if way == "fwd":
            r, y = kda.add_norm_fwd(st["r"], st["x"], st["w"], alpha=st["alpha"], eps=EPS)
            return dict(r=r, y=y)
        grads = kda.add_norm_bwd(st["r"], st["w"], st["dy"], st["dr"], x=st["x"], alpha=st["alpha"], eps=EPS)
        return {k: v for k, v in grads.items() if v is not None}
    if way == "fwd":
        x8 = kda.pack8(st["x"])
        return dict(code=x8.codes, e=x8.scales)
    return dict(x=kda.unpack8(st["x8"], TYPES[c["t"]]))


def _plain(st, c):
    op, way = c["op"], c.get("way")
    if op == "step":
        a = st["g"].float().exp()
        x = st["x"].float()
        h = a * st["h"] + (-torch.expm1(st["g"].float()) * x if c["tied"] else x)
        return dict(o=h.to(st["x"].dtype), h=h)
    if op == "scan":
        return _plain_scan(st, c) if way == "fwd" else _plain_scan_bwd(st, c)
    if op == "gated":
        return _plain_gated(st, c) if way == "fwd" else _plain_gated_bwd(st, c)
    if op == "add":
        return _plain_add(st, c) if way == "fwd" else _plain_add_bwd(st, c)
    if way == "fwd":
        code, e = _plain_pack(st["x"])
        return dict(code=code, e=e)
    return dict(x=_plain_unpack(st["code"], st["e"]).to(TYPES[c["t"]]))


def _linear(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling."""
    d = 1
    while d < b.shape[1]:
        b = torch.cat([b[:, :d], torch.addcmul(b[:, d:], a[:, d:], b[:, :-d])], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _starts(st, c):
    """First and last tokens of the sequences that have any, as (rows of [B * T], sequences)."""
    cu = st["cu"].long()
    some = (cu[1:] > cu[:-1]).nonzero()[:, 0]
    return cu[some], cu[some + 1] - 1, some


def _plain_h(st, c):
    """States after and before every token, [B, T, C] in 32 bits."""
    B, T, C = st["x"].shape
    g, x = st["g"].float(), st["x"].float()
    a, b = g.exp(), -torch.expm1(g) * x if c["tied"] else x.clone()
    first, _, seq = _starts(st, c)
    a, b = a.view(-1, C), b.view(-1, C)
    if st["h0"] is not None:
        b[first] += a[first] * st["h0"][seq]
    a[first] = 0.0
    h = _linear(a.view(B, T, C), b.view(B, T, C)).view(-1, C)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = 0.0 if st["h0"] is None else st["h0"][seq]
    return h.view(B, T, C), before.view(B, T, C)


def _ends(st, empty):
    """A state for every sequence: ``empty`` (or zeros) where it has no token."""
    n, C = st["cu"].shape[0] - 1, st["x"].shape[2]
    return torch.zeros(n, C, device=DEV) if empty is None else empty.clone()


def _plain_scan(st, c):
    h, _ = _plain_h(st, c)
    _, last, seq = _starts(st, c)
    ht = _ends(st, st["h0"])
    ht[seq] = h.view(-1, c["C"])[last]
    return dict(o=h.to(st["x"].dtype), ht=ht)


def _plain_scan_bwd(st, c):
    B, T, C = st["x"].shape
    _, before = _plain_h(st, c)
    g, x, do = st["g"].float(), st["x"].float(), st["do"].float().clone()
    a = g.exp()
    first, last, seq = _starts(st, c)
    if st["dht"] is not None:
        do.view(-1, C)[last] += st["dht"][seq]
    # l_t = do_t + a_{t+1} l_{t+1}: the same recurrence from the other end
    nxt = torch.cat([a.view(-1, C)[1:], torch.zeros(1, C, device=DEV)])
    nxt[last] = 0.0
    lam = _linear(nxt.view(B, T, C).flip(1), do.flip(1)).flip(1)
    m = a * lam
    dx = -torch.expm1(g) * lam if c["tied"] else lam
    dg = m * (before - x) if c["tied"] else m * before
    out = dict(dx=dx.to(st["x"].dtype), dg=dg.to(st["x"].dtype))
    if st["h0"] is not None:
        out["dh0"] = _ends(st, st["dht"])
        out["dh0"][seq] = m.view(-1, C)[first]
    return out


def _gate(z, act):
    """s(z) and s'(z)."""
    s = 1.0 / (1.0 + torch.exp(-z))
    return (s, s * (1.0 - s)) if act == "sigmoid" else (z * s, s * (1.0 + z * (1.0 - s)))


def _plain_gated(st, c):
    x, z = st["x"].float(), st["z"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = (x * r * st["w"] * _gate(z, c["act"])[0]).to(st["x"].dtype)
    if not c["keep"]:
        return dict(y=y)
    (xc, xe), (zc, ze) = _plain_pack(st["x"]), _plain_pack(st["z"])
    return dict(y=y, xc=xc, xe=xe, zc=zc, ze=ze)


def _plain_gated_bwd(st, c):
    x, z = st["x"], st["z"]
    if c["keep"]:
        x, z = _plain_unpack(*st["x8"]), _plain_unpack(*st["z8"])
    x, z, dy = x.float(), z.float(), st["dy"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    s, ds = _gate(z, c["act"])
    n = x * r
    dn = dy * st["w"] * s
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    t = st["dy"].dtype
    return dict(dx=dx.to(t), dgate=(dy * n * st["w"] * ds).to(t), dw=(dy * n * s).flatten(0, 1).sum(0))


def _plain_add(st, c):
    x = st["x"].float()
    r = st["r"].float() + (x if st["alpha"] is None else st["alpha"] * x)
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * st["w"]
    return dict(r=r.to(st["r"].dtype), y=y.to(st["x"].dtype))


def _plain_add_bwd(st, c):
    r, dy = st["r"].float(), st["dy"].float()
    inv = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    n, dn = r * inv, dy * st["w"]
    dr = st["dr"].float() + inv * (dn - n * (dn * n).mean(-1, keepdim=True))
    dx = dr if st["alpha"] is None else st["alpha"] * dr
    out = dict(dres=dr.to(st["r"].dtype), dx=dx.to(st["x"].dtype), dw=(dy * n).sum(0))
    if c["alpha"] == "vector":
        out["dalpha"] = (dr * st["x"].float()).sum(0)
    return out


def _plain_pack(x):
    n = x.shape[-1]
    v = x.float()
    if n % BLOCK:
        v = torch.nn.functional.pad(v, (0, BLOCK - n % BLOCK))
    v = v.unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1)
    # top = f * 2^k with f in [0.5, 1): 448 = 0.875 * 2^9
    f, k = torch.frexp(top)
    e = torch.where(top > 0, k - 9 + (f > 0.875), -126).clamp(min=-126)
    code = torch.ldexp(v, -e.unsqueeze(-1)).flatten(-2)[..., :n].to(E4M3)
    return code.contiguous(), (e + 127).to(torch.uint8)


def _plain_unpack(code, e):
    scale = torch.ldexp(torch.ones_like(e, dtype=F32), e.int() - 127)
    return code.float() * scale.repeat_interleave(BLOCK, -1)[..., :code.shape[-1]]


# ---- floors --------------------------------------------------------------------------------

def work(case):
    c, e = case, 2 if case["t"] == "bf16" else 4
    op, way = c["op"], c.get("way")
    if op == "step":
        n = c["B"] * c["C"]
        return dict(bytes=n * (3 * e + 8), flops=4 * n)
    if op == "scan":
        n, states = c["B"] * c["T"] * c["C"], (c["seqs"] or c["B"]) * c["C"] * 4
        if way == "fwd":
            return dict(bytes=3 * e * n + states * (2 if c["h0"] else 1), flops=4 * n)
        return dict(bytes=5 * e * n + (states * 3 if c["h0"] else 0), flops=10 * n)
    if op == "gated":
        n, w = c["T"] * c["H"] * c["D"], c["D"] * 4
        kept = 2 * (n + c["T"] * c["H"] * -(-c["D"] // BLOCK)) if c["keep"] else 0
        if way == "fwd":
            return dict(bytes=3 * e * n + kept + w, flops=10 * n)
        return dict(bytes=3 * e * n + (kept or 2 * e * n) + 2 * w, flops=24 * n)
    n = c["T"] * c["D"]
    if op == "add":
        re = 2 if c["res"] == "bf16" else 4
        vec = c["D"] * 4 * (2 if c["alpha"] == "vector" else 1)
        if way == "fwd":
            return dict(bytes=n * (2 * re + 2 * e) + vec, flops=6 * n)
        # without a scale the two gradients are one, where their types agree
        dx = 0 if c["alpha"] == "none" and re == e else e
        x = e if c["alpha"] == "vector" else 0
        return dict(bytes=n * (3 * re + e + dx + x) + 2 * vec, flops=14 * n)
    return dict(bytes=n * (e + 1) + c["T"] * -(-c["D"] // BLOCK), flops=2 * n)


# ---- the definition in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    c, st = case, prepare(case, seed)
    op, way = c["op"], c.get("way")
    if op == "step":
        a = st["g"].double().exp()
        h = a * st["h"].double() + ((1 - a) if c["tied"] else 1) * st["x"].double()
        return dict(o=h, h=h)
    if op == "scan":
        return _exact_scan(st, c)
    if op == "pack":
        code, e = _exact_pack(st["x"])
        return dict(code=code, e=None) if way == "fwd" else dict(x=_held(st["x"]))
    if op == "gated":
        x, z, w = st["x"].double(), st["z"].double(), st["w"].double()
        if way == "fwd":
            s = torch.sigmoid(z) * (z if c["act"] == "silu" else 1)
            y = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w * s
            if not c["keep"]:
                return dict(y=y)
            return dict(y=y, xc=_exact_pack(st["x"])[0], xe=None, zc=_exact_pack(st["z"])[0], ze=None)
        if c["keep"]:
            x, z = _held(st["x"]), _held(st["z"])
        x, z, w = x.requires_grad_(), z.requires_grad_(), w.requires_grad_()
        s = torch.sigmoid(z) * (z if c["act"] == "silu" else 1)
        y = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w * s
        dx, dz, dw = torch.autograd.grad(y, (x, z, w), st["dy"].double())
        return dict(dx=dx, dgate=dz, dw=dw)
    r, x, w = st["r"].double(), st["x"].double(), st["w"].double()
    alpha = st["alpha"].double() if c["alpha"] == "vector" else 1.0 if st["alpha"] is None else st["alpha"]
    if way == "fwd":
        r = r + alpha * x
        return dict(r=r, y=w * r / (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt())
    r, w = r.requires_grad_(), w.requires_grad_()
    y = w * r / (r.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    dr, dw = torch.autograd.grad(y, (r, w), st["dy"].double())
    dr = dr + st["dr"].double()
    out = dict(dres=dr, dx=alpha * dr, dw=dw)
    if c["alpha"] == "vector":
        out["dalpha"] = (dr * x).sum(0)
    return out


def _exact_pack(x):
    """x / 2^e before its rounding to a code, and 2^e, with the exponent found by trying it."""
    n, v = x.shape[-1], x.double()
    pad = torch.zeros(*x.shape[:-1], -n % BLOCK, dtype=torch.float64, device=DEV)
    v = torch.cat([v, pad], -1).unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    e = (top.clamp(min=1e-300) / 448).log2().ceil() - 1
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp(min=-126)
    return (v / torch.exp2(e)).flatten(-2)[..., :n], torch.exp2(e)


def _held(x):
    """The values that the kept codes of x stand for."""
    v, s = _exact_pack(x)
    s = s.expand(*s.shape[:-1], BLOCK).flatten(-2)[..., :x.shape[-1]]
    return v.float().to(E4M3).double() * s


def _exact_scan(st, c):
    """One token after the other, over all the sequences of a batch at once."""
    B, T, C = st["x"].shape
    cu = st["cu"].tolist()
    firsts = {a: i for i, (a, b) in enumerate(zip(cu, cu[1:])) if b > a}
    lasts = {b - 1: i for i, (a, b) in enumerate(zip(cu, cu[1:])) if b > a}
    h0 = None if st["h0"] is None else st["h0"].double()
    packed = bool(c["seqs"])
    a = st["g"].double().exp()
    x = st["x"].double()
    put = -torch.expm1(st["g"].double()) * x if c["tied"] else x
    o, before = torch.empty_like(x), torch.empty_like(x)
    ht = _ends(st, st["h0"]).double()
    h = torch.zeros(B, C, dtype=torch.float64, device=DEV)
    if not packed and h0 is not None:
        h = h0
    for t in range(T):
        if packed and t in firsts:
            h = torch.zeros_like(h) if h0 is None else h0[firsts[t]][None]
        before[:, t] = h
        h = torch.addcmul(put[:, t], a[:, t], h)
        o[:, t] = h
        if packed and t in lasts:
            ht[lasts[t]] = h[0]
    if c["way"] == "fwd":
        return dict(o=o, ht=ht if packed else h)
    dht = None if st["dht"] is None else st["dht"].double()
    lam, do = torch.empty_like(x), st["do"].double()
    dh0 = _ends(st, st["dht"]).double()
    m = torch.zeros(B, C, dtype=torch.float64, device=DEV)
    if not packed and dht is not None:
        m = dht
    for t in reversed(range(T)):
        if packed and t in lasts:
            m = torch.zeros_like(m) if dht is None else dht[lasts[t]][None]
        lam[:, t] = do[:, t] + m
        m = a[:, t] * lam[:, t]
        if packed and t in firsts:
            dh0[firsts[t]] = m[0]
    out = dict(dx=-torch.expm1(st["g"].double()) * lam if c["tied"] else lam,
               dg=a * lam * (before - x if c["tied"] else before))
    if h0 is not None:
        out["dh0"] = dh0 if packed else m
    return out
