"""Cases of the paged key-value cache operators: appending tokens, attention of one new token
per sequence, attention of prompt tokens, and the page bookkeeping (fork, extend, free, compact).

Each case has a plain form in elementary torch operations (``own`` false), the framework's
calls (``own`` true) and a 64-bit evaluation of the operator's definition (``exact``).

Definitions, for sequence s with ``kv_lens[s]`` tokens in the cache, token j of it in row
``j % page_size`` of page ``block_table[s, j // page_size]``, and query head h reading key head
``h // (HQ / HKV)``:

    visible(p, j) = j <= p and (window == 0 or j > p - window or j < sinks)
    o = sum_j softmax_j(scale q . k_j over the visible j) v_j       (zeros if none is visible)
    lse = log sum_j exp(scale q . k_j)                              (-inf if none is visible)

The query of a decode call stands at p = kv_lens[s] - 1; token i of the n_s query tokens of a
prompt call at p = kv_lens[s] - n_s + i.  A page is free when its reference count is 0.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ---- the cases -----------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch of 256 sequences writes one token per sequence and layer
        dict(name="append_step", op="append", S=256, lo=1, hi=8192, salt=1, new="one", HKV=4, D=128,
             page=64, kv="bf16"),
        # five long prompts enter an 8-bit cache, 32k tokens in all
        dict(name="append_prompts_e4m3", op="append", S=5, lo=3000, hi=11000, salt=2, new="all",
             HKV=8, D=128, page=64, kv="e4m3"),
        # a single user's next token: latency alone
        dict(name="decode_one", op="decode", S=1, lo=777, hi=777, salt=0, HQ=16, HKV=4, D=128,
             page=16, kv="bf16", window=0, sinks=0),
        # a serving batch with very unequal lengths up to the 8192-token context
        dict(name="decode_batch", op="decode", S=64, lo=200, hi=8192, salt=3, HQ=16, HKV=4, D=128,
             page=64, kv="bf16", window=0, sinks=0),
        # three users with long documents and an 8-bit cache: few rows, long axis
        dict(name="decode_long_e4m3", op="decode", S=3, lo=60000, hi=131072, salt=4, HQ=64, HKV=8,
             D=128, page=128, kv="e4m3", window=0, sinks=0),
        # a batch on a window layer: the last 1024 tokens and the first four
        dict(name="decode_window", op="decode", S=128, lo=50, hi=16384, salt=5, HQ=32, HKV=8, D=64,
             page=32, kv="bf16", window=1024, sinks=4),
        # short prompts of a chat arriving together, heads of 64 without sharing
        dict(name="prefill_short", op="prefill", S=4, qlo=1, qhi=200, ctx=0, salt=6, HQ=8, HKV=8,
             D=64, page=16, kv="bf16", window=0, sinks=0),
        # one prompt that fills the 8192-token context
        dict(name="prefill_context", op="prefill", S=1, qlo=8192, qhi=8192, ctx=0, salt=7, HQ=16,
             HKV=4, D=128, page=64, kv="bf16", window=0, sinks=0),
        # the next chunks of two long documents on a window layer with an 8-bit cache
        dict(name="prefill_window_e4m3", op="prefill", S=2, qlo=1700, qhi=2048, ctx=14000, salt=8,
             HQ=16, HKV=4, D=128, page=128, kv="e4m3", window=4096, sinks=4),
        # four continuations sampled from one prompt, six attention layers (K and V pools each)
        dict(name="fork_few", op="fork", S=32, live=3, lo=100, hi=4000, children=4, salt=9, pools=12,
             pages=512, HKV=4, D=128, page=64),
        # a wide beam: 128 children at once
        dict(name="fork_beam", op="fork", S=512, live=48, lo=100, hi=8192, children=128, salt=10,
             pools=12, pages=4096, HKV=2, D=128, page=64),
        # half of the sequences have ended: release them and close the holes
        dict(name="free_compact", op="compact", S=96, live=96, lo=100, hi=3000, drop=48, salt=11,
             pools=4, pages=2560, HKV=4, D=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random())) if hi > lo else lo


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "fork", "compact"])
    salt, D, page = rng.randrange(1000), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    HKV = rng.choice([1, 2, 4, 8])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log_int(rng, 100, 4096), rng.randrange(0, 9))])
    if op == "append":
        new = rng.choice(["one", "all"])
        S = _log_int(rng, 1, 256) if new == "one" else _log_int(rng, 1, 8)
        hi = _log_int(rng, 200, 8192) if new == "one" else _log_int(rng, 200, 32768 // S)
        return dict(op=op, S=S, lo=max(1, hi // 8), hi=hi, salt=salt, new=new, HKV=HKV, D=D,
                    page=page, kv=kv)
    G = rng.choice([1, 2, 3, 4, 5, 8])
    if op == "decode":
        S = _log_int(rng, 1, 128)
        hi = _log_int(rng, 100, min(131072, (1 << 19) // S // HKV * 2))
        return dict(op=op, S=S, lo=max(1, hi // 16), hi=hi, salt=salt, HQ=HKV * G, HKV=HKV, D=D,
                    page=page, kv=kv, window=window, sinks=sinks)
    if op == "prefill":
        S = rng.choice([1, 1, 2, 3, 4])
        ctx = rng.choice([0, 0, _log_int(rng, 10, 14000)])
        qhi = _log_int(rng, 5, 4096 if S == 1 and ctx == 0 else 1024)
        HKV = min(HKV, 16 // G) if G <= 16 else 1
        return dict(op=op, S=S, qlo=max(1, qhi // 4), qhi=qhi, ctx=ctx, salt=salt, HQ=HKV * G,
                    HKV=HKV, D=D, page=page, kv=kv, window=window, sinks=sinks)
    pools, live = rng.choice([2, 4, 8, 12]), _log_int(rng, 2, 64)
    hi = _log_int(rng, 50, 3000)
    HKV = min(HKV, 4)
    c = dict(op=op, live=live, lo=max(1, hi // 8), hi=hi, salt=salt, pools=pools, HKV=HKV, D=D,
             page=page)
    held = sum(-(-n // page) for n in _lens(c, live))
    if op == "fork":
        n = _log_int(rng, 1, 64)
        return c | dict(S=live + n + rng.randrange(5), children=n, pages=held + 2 * n + live + rng.randrange(9))
    return c | dict(S=live, drop=rng.randrange(1, live), pages=held + rng.randrange(1, 200))


def _spread(n, lo, hi, salt):
    """n lengths in [lo, hi], spread over their logarithm by golden-ratio steps."""
    u = [(0.137 * salt + 0.6180339887498949 * (i + 1)) % 1.0 for i in range(n)]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** x)))) for x in u]


def _lens(c, n):
    return _spread(n, c["lo"], c["hi"], c["salt"])


def _shape(c):
    """Tokens in the cache and query (or new) tokens of each sequence."""
    if c["op"] == "prefill":
        q = _spread(c["S"], c["qlo"], c["qhi"], c["salt"])
        old = _spread(c["S"], max(1, c["ctx"] // 2), c["ctx"], c["salt"] + 1) if c["ctx"] else [0] * c["S"]
        return [a + b for a, b in zip(q, old)], q
    kv = _lens(c, c["S"])
    return kv, (kv if c.get("new") == "all" else [1] * c["S"])


def _parents(c):
    return [(c["salt"] + 3 * i) % c["live"] for i in range(c["children"])]


def _dropped(c):
    """Ended sequences, spread over the slots."""
    return sorted(range(c["live"]), key=lambda i: (0.6180339887498949 * (i + c["salt"])) % 1.0)[:c["drop"]]


# ---- inputs --------------------------------------------------------------------------------

def _randn(gen, *shape, dtype=BF16):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)


def _pool(gen, c, pages):
    """One pool [pages, page, HKV, D] in the cache's type, and its scale per head."""
    x = _randn(gen, pages, c["page"], c["HKV"], c["D"])
    if c.get("kv", "bf16") == "bf16":
        return x, None
    s = (1.0 + torch.rand(c["HKV"], generator=gen, device=DEV)) * 0.01
    return (x.float() / s[:, None]).clamp(-448, 448).to(E4M3), s


def _table(gen, rows, width, lens, page, pages):
    """A block table whose pages lie in no order, -1 where a sequence has no page."""
    held = [-(-n // page) for n in lens]
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = perm[at:at + h]
        at += h
    return table


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(c=c)
    if c["op"] in ("fork", "compact"):
        lens = _lens(c, c["live"])
        width = max(-(-(n + 1) // c["page"]) for n in lens)
        table = _table(gen, c["S"], width, lens, c["page"], c["pages"])
        refs = torch.zeros(c["pages"], dtype=torch.int32, device=DEV)
        used = table[table >= 0].long()
        refs[used] = 1
        st.update(table=table, lens=_ints(lens + [0] * (c["S"] - c["live"])), refs=refs,
                  pools=[_randn(gen, c["pages"], c["page"], c["HKV"], c["D"]) for _ in range(c["pools"])])
        if c["op"] == "fork":
            n = c["children"]
            st["parents"] = _ints(_parents(c))
            free_rows = torch.randperm(c["S"] - c["live"], generator=gen, device=DEV)[:n]
            st["children"] = (free_rows + c["live"]).to(torch.int32)
        else:
            st["slots"] = _ints(_dropped(c))
        if own:
            import gated_delta_rule_41_gb300 as kda
            st["kda"] = kda
            st["book"] = kda.PageBook(c["pages"], c["page"], st["pools"])
        return st
    kv, qn = _shape(c)
    held = sum(-(-n // c["page"]) for n in kv)
    pages = held + max(2, held // 8)
    width = -(-max(kv) // c["page"])
    st["k"], st["ks"] = _pool(gen, c, pages)
    st["v"], st["vs"] = _pool(gen, c, pages)
    st["table"] = _table(gen, c["S"], width, kv, c["page"], pages)
    st["lens"] = _ints(kv)
    T = sum(qn)
    cu = [0]
    for n in qn:
        cu.append(cu[-1] + n)
    st["cu"] = _ints(cu)
    st["max_q"] = max(qn)
    if c["op"] == "append":
        # the new keys and values are slices of one projection's output
        qkv = _randn(gen, T, 2 * c["HKV"], c["D"])
        st["nk"], st["nv"] = qkv[:, :c["HKV"]], qkv[:, c["HKV"]:]
    else:
        st["q"] = 2.0 * _randn(gen, T, c["HQ"], c["D"])
        st["scale"] = c["D"] ** -0.5
    if own:
        import gated_delta_rule_41_gb300 as kda
        st["kda"] = kda
        st["kvp"] = kda.KVPages(st["k"], st["v"], k_scale=st["ks"], v_scale=st["vs"])
        if c["op"] == "decode":
            st["ws"] = kda.paged_decode_workspace(st["kvp"], c["S"], c["HQ"])
        elif c["op"] == "prefill":
            st["ws"] = kda.paged_prefill_workspace(st["kvp"], c["S"], T, c["HQ"])
    return st


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    st, c = state, state["c"]
    if own:
        kda = st["kda"]
        if c["op"] == "append":
            kda.paged_append(st["kvp"], st["nk"], st["nv"], st["table"], st["lens"],
                             None if c["new"] == "one" else st["cu"])
            return dict(k=st["k"], v=st["v"])
        if c["op"] == "decode":
            o, lse = kda.paged_decode(st["q"], st["kvp"], st["table"], st["lens"], scale=st["scale"],
                                      window=c["window"], sinks=c["sinks"], workspace=st["ws"],
                                      return_lse=True)
            return dict(o=o, lse=lse)
        if c["op"] == "prefill":
            o, lse = kda.paged_prefill(st["q"], st["kvp"], st["table"], st["lens"], st["cu"],
                                       scale=st["scale"], window=c["window"], sinks=c["sinks"],
                                       workspace=st["ws"], return_lse=True)
            return dict(o=o, lse=lse)
        table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
        if c["op"] == "fork":
            st["book"].fork(st["parents"], st["children"], table, lens, refs)
            st["book"].extend(1, table, lens, refs)
        else:
            st["book"].free(st["slots"], table, lens, refs)
            st["book"].compact(table, lens, refs)
        return dict(table=table, lens=lens, refs=refs, pools=st["pools"])
    if c["op"] == "append":
        return _plain_append(st, c)
    if c["op"] == "decode":
        return _plain_attention(st, c, st["q"][:, None], torch.ones_like(st["lens"]))
    if c["op"] == "prefill":
        n = st["cu"][1:] - st["cu"][:-1]
        i = torch.arange(st["max_q"], device=DEV)
        at = (st["cu"][:-1, None] + i).clamp(max=st["q"].shape[0] - 1).long()
        return _plain_attention(st, c, st["q"][at], n, at)
    return _plain_fork(st, c) if c["op"] == "fork" else _plain_compact(st, c)


def _plain_append(st, c):
    T = st["nk"].shape[0]
    t = torch.arange(T, device=DEV)
    s = t if c["new"] == "one" else (t[:, None] >= st["cu"][None, 1:]).sum(1)
    ends = t + 1 if c["new"] == "one" else st["cu"].long()[s + 1]
    pos = st["lens"].long()[s] - (ends - t)
    page = st["table"][s, (pos // c["page"])].long()
    row = pos % c["page"]
    if c["kv"] == "bf16":
        st["k"][page, row], st["v"][page, row] = st["nk"], st["nv"]
    else:
        st["k"].view(torch.uint8)[page, row] = _quant(st["nk"], st["ks"]).view(torch.uint8)
        st["v"].view(torch.uint8)[page, row] = _quant(st["nv"], st["vs"]).view(torch.uint8)
    return dict(k=st["k"], v=st["v"])


def _quant(x, s):
    """e4m3 codes of x / s, with the reciprocal of s rounded first; out of range saturates."""
    return (x.float() * (1.0 / s)[:, None]).clamp(-448, 448).to(E4M3)


def _rows(pool, s, table):
    """The cache rows of every sequence, [S, width * page, HKV, D] in 32 bits."""
    at = table.clamp(min=0).long()
    x = (pool.view(torch.uint8)[at].view(E4M3) if pool.dtype == E4M3 else pool[at]).float()
    x = x.flatten(1, 2)
    return x if s is None else x * s[:, None]


def _plain_attention(st, c, q, n, at=None):
    """q [S, M, HQ, D], n[s] of the M rows of sequence s in use."""
    S, M, HQ, D = q.shape
    G = HQ // c["HKV"]
    k, v = _rows(st["k"], st["ks"], st["table"]), _rows(st["v"], st["vs"], st["table"])
    j = torch.arange(k.shape[1], device=DEV)
    p = (st["lens"] - n)[:, None] + torch.arange(M, device=DEV)               # [S, M]
    see = j <= p[..., None]
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    qg = (q.float() * st["scale"]).view(S, M, c["HKV"], G, D).permute(0, 2, 3, 1, 4)  # [S,HKV,G,M,D]
    x = torch.matmul(qg.flatten(2, 3), k.permute(0, 2, 3, 1))                 # [S,HKV,G*M,L]
    x = x.view(S, c["HKV"], G, M, -1).masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3)).view(S, c["HKV"], G, M, D)
    o = torch.where(total > 0, o / total.clamp(min=1e-30), torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, M, HQ, D).to(q.dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(S, M, HQ)
    if at is None:
        return dict(o=o[:, 0], lse=lse[:, 0])
    T = st["q"].shape[0]
    flat = torch.arange(T, device=DEV)
    s = (flat[:, None] >= st["cu"][None, 1:]).sum(1)
    i = flat - st["cu"].long()[s]
    return dict(o=o[s, i], lse=lse[s, i])


def _take(refs, want, table, rows, first):
    """The lowest free pages, in order: want[i] of them into table[rows[i], first[i]:]."""
    free = torch.argsort((refs > 0).to(torch.int32), stable=True)
    before = want.cumsum(0) - want
    col = torch.arange(table.shape[1], device=DEV)
    off = col - first[:, None]
    new = (off >= 0) & (off < want[:, None])
    page = free[(before[:, None] + off).clamp(0, refs.numel() - 1)]
    table[rows] = torch.where(new, page.to(torch.int32), table[rows])
    refs.scatter_add_(0, page.flatten(), new.flatten().to(torch.int32))
    return new, page


def _plain_fork(st, c):
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    par, ch, P = st["parents"].long(), st["children"].long(), c["page"]
    n = lens[par].long()
    full, part = n // P, n % P != 0
    row, col = table[par], torch.arange(table.shape[1], device=DEV)
    shared = col < full[:, None]
    table[ch] = torch.where(shared, row, torch.full_like(row, -1))
    _, page = _take(refs, part.long(), table, ch, full)
    refs.scatter_add_(0, row.clamp(min=0).flatten().long(), shared.flatten().to(torch.int32))
    lens[ch] = lens[par]
    last = full.clamp(max=table.shape[1] - 1)[:, None]
    src = row.gather(1, last)[:, 0].long().clamp(min=0)
    dst = torch.where(part, table[ch].gather(1, last)[:, 0].long(), src)
    pools = [pool.index_copy_(0, dst, pool[src]) for pool in st["pools"]]
    # the next token of every live sequence
    grown = torch.where(lens > 0, lens + 1, lens).long()
    held = (lens.long() + P - 1) // P
    _take(refs, (grown + P - 1) // P - held, table, torch.arange(lens.numel(), device=DEV), held)
    lens.copy_(grown)
    return dict(table=table, lens=lens, refs=refs, pools=pools)


def _plain_compact(st, c):
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    slots = st["slots"].long()
    row = table[slots].flatten().long()
    refs.scatter_add_(0, row.clamp(min=0), -(row >= 0).to(torch.int32))
    table[slots], lens[slots] = -1, 0
    # live pages at or above their number move, in order, into the holes below it
    live, ids = refs > 0, torch.arange(refs.numel(), device=DEV)
    top = ids >= live.sum()
    src, dst = (live & top).nonzero()[:, 0], (~live & ~top).nonzero()[:, 0]
    pools = [_moved(pool, src, dst) for pool in st["pools"]]
    to = ids.to(torch.int32)
    to[src] = dst.to(torch.int32)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], table)
    refs[dst] = refs[src]
    refs[src] = 0
    return dict(table=table, lens=lens, refs=refs, pools=pools)


def _moved(pool, src, dst):
    pool[dst] = pool[src]
    return pool


# ---- floors --------------------------------------------------------------------------------

def _seen(c, p):
    """Tokens that a query at position p sees."""
    if not c["window"] or p + 1 <= c["window"]:
        return max(0, p + 1)
    return c["window"] + min(c["sinks"], p + 1 - c["window"])


def work(case):
    c = case
    e = 2 if c.get("kv", "bf16") == "bf16" else 1
    row = c["HKV"] * c["D"]
    if c["op"] == "append":
        T = sum(_shape(c)[1])
        return dict(bytes=2 * T * row * (2 + e) + 8 * c["S"], flops=0 if e == 2 else 2 * T * row)
    if c["op"] in ("decode", "prefill"):
        kv, qn = _shape(c)
        read = pairs = 0
        for L, n in zip(kv, qn):
            first = L - n
            low = max(0, first + 1 - c["window"]) if c["window"] else 0
            read += L - low + min(c["sinks"], low)
            pairs += sum(_seen(c, p) for p in range(first, L))
        pages = sum(-(-n // c["page"]) for n in kv)
        io = sum(qn) * c["HQ"] * (4 * c["D"] + 4) + 4 * pages + 8 * c["S"]
        return dict(bytes=2 * read * row * e + io, flops=4 * pairs * c["HQ"] * c["D"])
    lens = _lens(c, c["live"])
    width = max(-(-(n + 1) // c["page"]) for n in lens)
    book = 2 * 4 * (c["S"] * width + c["S"] + c["pages"])
    page = c["pools"] * c["page"] * row * 2
    if c["op"] == "fork":
        return dict(bytes=2 * page * sum(lens[p] % c["page"] != 0 for p in _parents(c)) + book, flops=0)
    gone = set(_dropped(c))
    left = sum(-(-n // c["page"]) for i, n in enumerate(lens) if i not in gone)
    # pages lie in random order: this many of the live ones are expected above their number
    return dict(bytes=2 * page * left * (1 - left / c["pages"]) + book, flops=0)


# ---- the definition in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] in ("fork", "compact"):
        return None                                     # copies and whole numbers
    st = prepare(c, seed)
    kv, qn = _shape(c)
    P = c["page"]
    if c["op"] == "append":
        out = {}
        for name, new, scale in (("k", "nk", "ks"), ("v", "nv", "vs")):
            pool = st[name].double()
            at = 0
            for s, n in enumerate(qn):
                j = torch.arange(kv[s] - n, kv[s], device=DEV)
                x = st[new][at:at + n].double()
                if st[scale] is not None:
                    x = (x / st[scale].double()[:, None]).clamp(-448, 448)
                pool[st["table"][s].long()[j // P], j % P] = x
                at += n
            out[name] = pool
        return out
    G, o, lse, at = c["HQ"] // c["HKV"], [], [], 0
    if sum(n * L for n, L in zip(qn, kv)) * c["HQ"] * c["D"] > 3e12:
        return None
    for s, (n, L) in enumerate(zip(qn, kv)):
        pages = st["table"][s].long()[torch.arange(-(-L // P), device=DEV)]
        k = (st["k"].view(torch.uint8)[pages].view(st["k"].dtype)).double().flatten(0, 1)[:L]
        v = (st["v"].view(torch.uint8)[pages].view(st["v"].dtype)).double().flatten(0, 1)[:L]
        q = st["q"][at:at + n].double()
        j, p = torch.arange(L, device=DEV), torch.arange(L - n, L, device=DEV)[:, None]
        hidden = j > p
        if c["window"]:
            hidden = hidden | ((j <= p - c["window"]) & (j >= c["sinks"]))
        heads, tops = [], []
        for h in range(c["HQ"]):
            g = h // G
            kk = k[:, g] if st["ks"] is None else k[:, g] * st["ks"][g].double()
            vv = v[:, g] if st["vs"] is None else v[:, g] * st["vs"][g].double()
            x = (q[:, h] @ kk.T) / math.sqrt(c["D"])
            x = x.masked_fill(hidden, -math.inf)
            heads.append(torch.softmax(x, -1) @ vv)
            tops.append(torch.logsumexp(x, -1))
        o.append(torch.stack(heads, 1))
        lse.append(torch.stack(tops, 1))
        at += n
    return dict(o=torch.cat(o), lse=torch.cat(lse))
