"""Plain 64-bit reference of the paged key-value cache: attention from its
definition, the page bookkeeping as host loops, and the error bounds that the
kernels' number formats give."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn
PAGE_NAN = 0x7F


def make_cache(S_lens, page, HKV, D, dtype, seed, layout="rows", spare=3, poison=True,
               device="cuda"):
    """Pools, scales, table and lengths for sequences of the given lengths, the
    pages in random order.  ``poison``: every slot that holds no token is NaN.
    layout: "rows" [pages, rows, heads, D], "heads" (heads before rows) or
    "joint" (K and V in one tensor)."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in S_lens]
    pages = sum(held) + spare
    width = max(held + [1]) + 1
    table = torch.full((len(S_lens), width), -1, dtype=torch.int32)
    perm, at = torch.randperm(pages, generator=g).to(torch.int32), 0
    used = torch.zeros(pages, page, dtype=torch.bool)
    for s, h in enumerate(held):
        table[s, :h] = perm[at:at + h]
        for i in range(h):
            used[perm[at + i], :max(0, min(page, S_lens[s] - i * page))] = True
        at += h
    x = torch.randn(2, pages, page, HKV, D, generator=g)
    scales = None
    if dtype == E4M3:
        scales = 0.01 * (1 + torch.rand(2, HKV, generator=g))
        x = (x / scales[:, None, None, :, None]).clamp(-448, 448)
    x = x.to(dtype)
    if poison:
        raw = x.view(torch.uint8) if dtype == E4M3 else x
        raw[:, ~used] = PAGE_NAN if dtype == E4M3 else float("nan")
    x = x.to(device)
    if layout == "heads":
        x = x.transpose(2, 3).contiguous().transpose(2, 3)
    if layout == "joint":
        x = torch.stack((x[0], x[1]), 1).contiguous().transpose(0, 1)
    sc = (None, None) if scales is None else tuple(s.contiguous().to(device) for s in scales)
    return dict(k=x[0], v=x[1], ks=sc[0], vs=sc[1], table=table.to(device),
                lens=torch.tensor(S_lens, dtype=torch.int32, device=device))


def tokens_of(pool, scale, table, s, n):
    """The first n tokens of sequence s in 64 bits [n, HKV, D] on the CPU."""
    page = pool.shape[1]
    j = torch.arange(n)
    raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
    x = raw[table[s].long()[(j // page).to(table.device)], (j % page).to(table.device)]
    x = (x.view(E4M3) if pool.dtype == E4M3 else x).double().cpu()
    return x if scale is None else x * scale.double().cpu()[:, None]


def attend(q, k, v, p, scale, window, sinks):
    """q [n, HQ, D], k, v [L, HKV, D], positions p [n], all 64-bit.  Returns o,
    lse, and for the bounds A = sum_j w_j |v_j| and X = max_j scale sum_d |q k|."""
    n, HQ, D = q.shape
    L, HKV, _ = k.shape
    G = HQ // HKV
    j = torch.arange(L)
    see = j <= p[:, None]
    if window:
        see &= (j > p[:, None] - window) | (j < sinks)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = scale * torch.einsum("nhd,lhd->nhl", q, kk)
    x = x.masked_fill(~see[:, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.where(see[:, None], torch.exp(x - lse[..., None]), torch.zeros_like(x))
    X = torch.einsum("nhd,lhd->nhl", q.abs(), kk.abs()).masked_fill(~see[:, None], 0)
    X = abs(scale) * (X.amax(-1) if L else torch.zeros(n, HQ, dtype=torch.float64))
    return (torch.einsum("nhl,lhd->nhd", w, vv), lse,
            torch.einsum("nhl,lhd->nhd", w, vv.abs()), X)


def check_attention(o, lse, ref):
    """Element bounds.  Output: bf16 rounds by up to 2^-8 |o|, which is at most
    2^-9 |o| + 2^-9 A, since |o| <= A = sum w |v|.  Weights: what that leaves of
    2^-9 A (the kernels keep a weight to 2^-11 or better), and the error of
    their logits.  Logits: D <= 128 products summed in fp32, in any
    order and with truncation, are off by at most 128 * 2^-23 of the sum of
    magnitudes X, 2^-16 X; exp2 adds 2^-21.  All of it times A = sum w |v|, twice
    where the sum of the weights carries it too."""
    ro, rl, A, X = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    dead = torch.isinf(rl)
    assert (o[dead] == 0).all() and (lse[dead] == -math.inf).all()
    assert torch.isfinite(o).all() and torch.isfinite(lse[~dead]).all()
    logit = 2.0 ** -16 * X + 2.0 ** -20
    bound = 2.0 ** -9 * ro.abs() + (2.0 ** -9 + 2 * logit[..., None]) * 1.01 * A + 1e-30
    worst = ((o - ro).abs() / bound)[~dead]
    assert not worst.numel() or worst.max() <= 1, f"output off: {worst.max():.3g} of its bound"
    worst = ((lse - rl).abs() / (logit + 2.0 ** -22 * rl.abs()))[~dead]
    assert not worst.numel() or worst.max() <= 1, f"lse off: {worst.max():.3g} of its bound"


def ref_decode(q, c, scale, window=0, sinks=0):
    lens, out = c["lens"].cpu().tolist(), []
    for s, n in enumerate(lens):
        k, v = (tokens_of(c[x], c[x + "s"], c["table"], s, n) for x in ("k", "v"))
        out.append(attend(q[s:s + 1].double().cpu(), k, v, torch.tensor([n - 1]), scale, window,
                          sinks))
    return [torch.cat(x) for x in zip(*out)]


def ref_prefill(q, c, qn, scale, window=0, sinks=0):
    lens, out, at = c["lens"].cpu().tolist(), [], 0
    for s, (n, m) in enumerate(zip(lens, qn)):
        k, v = (tokens_of(c[x], c[x + "s"], c["table"], s, n) for x in ("k", "v"))
        out.append(attend(q[at:at + m].double().cpu(), k, v, torch.arange(n - m, n), scale, window,
                          sinks))
        at += m
    return [torch.cat(x) for x in zip(*out)]


class Book:
    """The page bookkeeping as host lists; pools are lists of per-page values."""

    def __init__(self, table, lens, refs, page, pools):
        self.table, self.lens, self.refs = table.tolist(), lens.tolist(), refs.tolist()
        self.page, self.pools = page, [p.clone() for p in pools]
        self.refused = False

    def _take(self, wants):
        """Page lists for each request, None where refused."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        out, at = [], 0
        for w in wants:
            at += w
            if w and at > len(free):
                self.refused = True
                out.append(None)
            else:
                out.append(free[at - w:at])
        for got in out:
            for p in got or []:
                self.refs[p] = 1
        return out

    def extend(self, add):
        pages = lambda n: -(-n // self.page)
        got = self._take([pages(n + a) - pages(n) for n, a in zip(self.lens, add)])
        for s, (g, a) in enumerate(zip(got, add)):
            if g is None:
                continue
            h = pages(self.lens[s])
            self.table[s][h:h + len(g)] = g
            self.lens[s] += a

    def fork(self, parents, children):
        got = self._take([int(self.lens[p] % self.page != 0) for p in parents])
        for p, c, g in zip(parents, children, got):
            if g is None:
                continue
            full = self.lens[p] // self.page
            row = self.table[p][:full]
            for x in row:
                self.refs[x] += 1
            if g:
                for pool in self.pools:
                    pool[g[0]] = pool[self.table[p][full]]
                row = row + g
            self.table[c] = row + [-1] * (len(self.table[c]) - len(row))
            self.lens[c] = self.lens[p]

    def free(self, slots):
        for s in slots:
            for x in self.table[s]:
                if x >= 0:
                    self.refs[x] -= 1
            self.table[s], self.lens[s] = [-1] * len(self.table[s]), 0

    def compact(self):
        L = sum(r > 0 for r in self.refs)
        src = [p for p in range(L, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(L) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            for pool in self.pools:
                pool[b] = pool[a]
        self.table = [[to.get(x, x) for x in row] for row in self.table]
