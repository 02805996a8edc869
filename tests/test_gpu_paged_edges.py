"""Paged key-value cache at its edges: refused calls, values and logits that
are not ordinary numbers, tables with released pages, streams and errors."""
import math

import pytest
import torch

import gated_delta_rule_41_gb300 as kda
from paged_util import (E4M3, check_attention, make_cache, ref_decode, ref_prefill,
                        tokens_of)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_41_gb300 import build
    build.build()


def kv(c):
    return kda.KVPages(c["k"], c["v"], k_scale=c["ks"], v_scale=c["vs"])


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rand_q(rows, HQ, D, seed, amp=2.0):
    g = torch.Generator().manual_seed(seed)
    return (amp * torch.randn(rows, HQ, D, generator=g)).to(BF16).cuda()


def widened(c, tokens):
    """The same cache with a table that could hold `tokens` tokens a row, so
    that calls of few query rows are split over the cached tokens."""
    cols = tokens // c["k"].shape[1]
    table = torch.full((c["table"].shape[0], cols), -1, dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = c["table"]
    return dict(c, table=table)


def rows_of(o, lse, ref, keep):
    """Outputs and reference of the chosen query rows."""
    keep = torch.as_tensor(keep)
    return o[keep.cuda()], lse[keep.cuda()], [x[keep] for x in ref]


# ---- refused calls ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("cu", [[0, 30, 20, 50], [0, 10, 20, 40], [1, 10, 20, 50],
                                [-3, 10, 20, 50]])
def test_refused_prompts_write_nothing_when_tokens_are_split(cu, dtype):
    c = widened(make_cache([50, 2000, 50], 16, 1, 64, dtype, 11), 4096)
    q = rand_q(50, 2, 64, 12)
    out = torch.full_like(q, 3.0)
    lse = torch.full((50, 2), 5.0, device="cuda")
    kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints(cu), out=out, lse=lse)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2
    assert (out == 3).all() and (lse == 5).all()
    # and the next call is as ever
    good = ints([0, 20, 40, 50])
    o, l = kda.paged_prefill(q, kv(c), c["table"], c["lens"], good, return_lse=True)
    kda.check()
    check_attention(o, l, ref_prefill(q, c, [20, 20, 10], 64 ** -0.5))


# ---- page counts that no book keeps ----

def test_compact_reports_negative_counts_and_stays_in_range():
    """A negative count is neither a holder nor a hole left over: the page counts as
    free, the held ones close up, and nothing else changes."""
    pages, g = 40, torch.Generator().manual_seed(50)
    pool = torch.randint(0, 1 << 15, (pages, 4, 4), generator=g, dtype=torch.int32).cuda()
    refs = torch.zeros(pages, dtype=torch.int32)
    held = [0, 2, 7, 8, 21, 30, 39]
    refs[held] = 1
    refs[[1, 3, 5, 25, 38]] = torch.tensor([-1, -3, -2 ** 31, -1, -7], dtype=torch.int32)
    table = torch.full((2, 5), -1, dtype=torch.int32)
    table[0, :3], table[1, :4] = torch.tensor(held[:3]), torch.tensor(held[3:])
    want_table, want_pool, want_refs = table.clone(), pool.clone(), refs.clone()
    n = len(held)
    to = dict(zip([p for p in held if p >= n], [p for p in range(n) if refs[p] <= 0]))
    for a, b in to.items():
        want_table[table == a] = b
        want_pool[b] = pool[a]
        want_refs[b], want_refs[a] = refs[a], 0
    dev = [table.cuda(), ints([12, 16]), refs.cuda()]
    book = kda.PageBook(pages, 4, [pool])
    book.compact(*dev)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2
    assert torch.equal(dev[0].cpu(), want_table) and torch.equal(dev[2].cpu(), want_refs)
    assert torch.equal(pool, want_pool)


# ---- NaN in queries and keys ----

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_decode_nan_query_or_keys_give_nan(dtype, D):
    """A NaN in a query, or in the key of an only token, is not an empty row."""
    c = make_cache([700, 40, 1, 0, 3000], 32, 2, D, dtype, 51)
    q = rand_q(5, 8, D, 52)
    q[0, 3, 5] = math.nan
    q[3, 0, 0] = math.nan                     # of a row that sees nothing
    k = c["k"].view(torch.uint8) if dtype == E4M3 else c["k"]
    k[c["table"][2, 0].item(), 0, 1] = 0x7F if dtype == E4M3 else math.nan
    o, lse = kda.paged_decode(q, kv(c), c["table"], c["lens"], return_lse=True)
    kda.check()
    assert o[0, 3].isnan().all() and lse[0, 3].isnan()
    assert o[2, 4:].isnan().all() and lse[2, 4:].isnan().all()
    assert (o[3] == 0).all() and (lse[3] == -math.inf).all()
    ref = ref_decode(torch.nan_to_num(q), c, D ** -0.5)
    heads = [0, 1, 2, 4, 5, 6, 7]
    check_attention(o[:1, heads], lse[:1, heads], [x[:1, heads] for x in ref])
    check_attention(o[2:3, :4], lse[2:3, :4], [x[2:3, :4] for x in ref])
    check_attention(*rows_of(o, lse, ref, [1, 4]))


@pytest.mark.parametrize("D,wide", [(64, 0), (128, 0), (128, 8192)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_prompt_nan_query_or_keys_give_nan(dtype, D, wide):
    lens, qn = [600, 1, 5], [300, 1, 9]       # the last one: four queries that see nothing
    c = make_cache(lens, 32, 2, D, dtype, 53)
    if wide:
        lens, qn = [6000, 1, 5], [3, 1, 9]
        c = widened(make_cache(lens, 32, 2, D, dtype, 53), wide)
    q = rand_q(sum(qn), 4, D, 54)
    bad = 1
    q[bad, 2, 7] = math.nan
    q[sum(qn[:2]), :, 0] = math.nan           # sees nothing
    k = c["k"].view(torch.uint8) if dtype == E4M3 else c["k"]
    k[c["table"][1, 0].item(), 0, 0] = 0x7F if dtype == E4M3 else math.nan
    cu = ints([0] + qn).cumsum(0).to(torch.int32)
    o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, return_lse=True)
    kda.check()
    assert o[bad, 2].isnan().all() and lse[bad, 2].isnan()
    one = qn[0]                               # the only token's key of head 0 is NaN
    assert o[one, :2].isnan().all() and lse[one, :2].isnan().all()
    assert (o[one + 1] == 0).all() and (lse[one + 1] == -math.inf).all()
    ref = ref_prefill(torch.nan_to_num(q), c, qn, D ** -0.5)
    check_attention(o[one:one + 1, 2:], lse[one:one + 1, 2:], [x[one:one + 1, 2:] for x in ref])
    check_attention(*rows_of(o, lse, ref, [i for i in range(sum(qn)) if i not in (bad, one)]))
    check_attention(o[bad:bad + 1, [0, 1, 3]], lse[bad:bad + 1, [0, 1, 3]],
                    [x[bad:bad + 1, [0, 1, 3]] for x in ref])


# ---- large logits ----

@pytest.mark.parametrize("amp", [3e3, 1.1e6, 1.7e6, 2.3e7, 1e9, 1e30])
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,qn", [([600], [600]), ([6000], [3])])
def test_equal_keys_weigh_the_same_at_logits_of_any_size(lens, qn, dtype, scale, amp):
    """All keys equal: o is the mean of the visible values, whatever the logit.
    Weights are equal but for their rounding, 2^-11 each, and the output is
    rounded to bf16: |o - mean| <= 2^-8 |mean| + 2^-10 mean |v|."""
    c = make_cache(lens, 32, 1, 128, dtype, 55, poison=False)
    c["k"].fill_(1.0)
    if c["ks"] is not None:
        c["ks"].fill_(1.0)
    q = torch.full((sum(qn), 2, 128), amp, dtype=BF16, device="cuda")
    cu = ints([0] + qn).cumsum(0).to(torch.int32)
    o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, scale=scale, return_lse=True)
    d, dl = kda.paged_decode(q[:1], kv(c), c["table"], c["lens"], scale=scale, return_lse=True)
    kda.check()
    ref = ref_prefill(q * 0, c, qn, 1.0)       # weights of one, in the reference too
    dref = ref_decode(q[:1] * 0, c, 1.0)
    top = scale * 128 * q[0, 0, 0].double().item()
    for x, l, r in ((o, lse, ref), (d, dl, dref)):
        bound = 2.0 ** -8 * r[0].abs() + 2.0 ** -10 * r[2]
        assert ((x.double().cpu() - r[0]).abs() <= bound).all()
        assert ((l.double().cpu() - (r[1] + top)).abs() <= 2.0 ** -21 * abs(top) + 1e-5).all()


# ---- a token that outweighs a long tail ----

@pytest.mark.parametrize("nats", [12.0, 16.6, 17.5])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("prefill", [False, True])
def test_small_weights_of_a_long_tail(prefill, dtype, nats):
    """The first token takes almost all of the weight and its value is zero: what
    is left is the tail's, all of one sign.  A weight is rounded by up to 2^-11 of
    itself (that is in the usual bound) or, where it is small, by 2^-32 of the
    largest: half of fp16's smallest step, 2^-25, with the largest at 2^7 or more.  The rows are many, so that no
    other CTA takes part of one."""
    n = 131072
    c = make_cache([n], 128, 2, 64, dtype, 56, poison=False)
    if c["ks"] is not None:
        c["ks"].fill_(1.0)
    c["k"].zero_()
    first = c["table"][0, 0].item()
    c["k"][first, 0, :, 0] = 1.0
    v = c["v"].view(torch.uint8) if dtype == E4M3 else c["v"].view(torch.int16)
    v &= 0x7F if dtype == E4M3 else 0x7FFF     # |v|: the tail adds up
    v[first, 0] = 0
    T = 8192 if prefill else 160
    q = torch.zeros(T, 4, 64, dtype=BF16, device="cuda")
    q[..., 0] = nats
    nats = q[0, 0, 0].item()
    if prefill:
        o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints([0, T]), scale=1.0,
                                   return_lse=True)
        o, lse, q = o[-2:], lse[-2:], q[-2:]
        ref = ref_prefill(q, c, [2], 1.0)
    else:
        table = c["table"].expand(T, -1).contiguous()
        o, lse = kda.paged_decode(q, kv(c), table, ints([n] * T), scale=1.0, return_lse=True)
        o, lse, q = o[:1], lse[:1], q[:1]
        ref = ref_decode(q, c, 1.0)
    kda.check()
    ro, rl, A, X = ref
    vmean = A.max() / (1 - math.exp(nats - rl.min().item()))     # mean |v| of the tail
    logit = 2.0 ** -16 * X + 2.0 ** -20
    bound = (2.0 ** -9 * ro.abs() + (2.0 ** -9 + 2 * logit[..., None]) * 1.01 * A
             + n * 2.0 ** -32 * vmean)
    worst = ((o.double().cpu() - ro).abs() / bound).max()
    assert worst <= 1, f"off: {worst:.3g} of its bound"
    assert ((lse.double().cpu() - rl).abs() <= logit + 2.0 ** -22 * rl.abs()).all()


# ---- values of unequal channels ----

@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("big", [1.0, 2.0 ** 20, 2.0 ** -40])
def test_channels_far_smaller_than_others(prefill, big):
    """Channels 2^-20 and 2^-30 of the others keep the precision that is stated:
    a value is rounded by up to 2^-37 of the largest |v|."""
    lens, qn = [700], [300]
    c = make_cache(lens, 32, 2, 128, BF16, 57, poison=False)
    c["v"].mul_(big)
    c["v"][..., 10:20] *= 2.0 ** -20
    c["v"][..., 30:40] *= 2.0 ** -30
    top = c["v"].abs().max().item()
    q = rand_q(300 if prefill else 1, 4, 128, 58)
    if prefill:
        o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints([0, 300]),
                                   return_lse=True)
        ref = ref_prefill(q, c, qn, 128 ** -0.5)
    else:
        o, lse = kda.paged_decode(q, kv(c), c["table"], c["lens"], return_lse=True)
        ref = ref_decode(q, c, 128 ** -0.5)
    kda.check()
    ro, rl, A, X = ref
    logit = 2.0 ** -16 * X + 2.0 ** -20
    bound = (2.0 ** -9 * ro.abs() + (2.0 ** -9 + 2 * logit[..., None]) * 1.01 * A
             + 2.0 ** -37 * top)
    for part in (slice(0, 10), slice(10, 20), slice(30, 40), slice(40, 128)):
        worst = ((o.double().cpu() - ro).abs() / bound)[..., part].max()
        assert worst <= 1, f"channels {part}: {worst:.3g} of the bound"


@pytest.mark.parametrize("big", [2.0 ** -110, 2.0 ** -125, 2.0 ** 110])
def test_values_at_the_ends_of_the_range(big):
    """The smallest values (some denormal) and the largest stay finite; what is below 2^-117
    may be rounded by 2^-125."""
    c = make_cache([400], 32, 1, 64, BF16, 76, poison=False)
    c["v"].copy_((c["v"].double() * big).to(BF16))
    q = rand_q(400, 2, 64, 77)
    o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints([0, 400]), return_lse=True)
    kda.check()
    ro, rl, A, X = ref_prefill(q, c, [400], 0.125)
    logit = 2.0 ** -16 * X + 2.0 ** -20
    bound = (2.0 ** -9 * ro.abs() + (2.0 ** -9 + 2 * logit[..., None]) * 1.01 * A + 2.0 ** -124)
    assert ((o.double().cpu() - ro).abs() <= bound).all()


# ---- infinities and NaN among values ----

VALUES = [math.nan, math.inf, -math.inf]


def poisoned(c, s, j, value, channel):
    v = c["v"].view(torch.uint8) if c["v"].dtype == E4M3 else c["v"]
    page = c["v"].shape[1]
    v[c["table"][s, j // page].item(), j % page, :, channel] = (
        0x7F if c["v"].dtype == E4M3 else value)


@pytest.mark.parametrize("kind", [(BF16, 0), (BF16, 1), (BF16, 2), (E4M3, 0)])
@pytest.mark.parametrize("heads", [(2, 2), (8, 2)])
@pytest.mark.parametrize("window,sinks,at", [(0, 0, (450,)), (0, 0, (3, 600, 699)), (100, 4, (50,)),
                                             (100, 4, (2, 500)), (300, 0, (0, 399, 400))])
@pytest.mark.parametrize("tokens", [700, 2100])
def test_values_reach_only_the_queries_that_see_them(tokens, window, sinks, at, heads, kind):
    """NaN and infinities in V, in one channel of some tokens: queries that see
    one get it, the others and the other channels are as ever."""
    dtype, which = kind
    n = 400 if tokens == 700 else 9           # 2100: split over the cached tokens
    at = [j + tokens - 700 if j > 60 else j for j in at]
    c = make_cache([tokens], 32, heads[1], 128, dtype, 59)
    if n == 9:
        c = widened(c, 8192)
    for j in at:
        poisoned(c, 0, j, VALUES[which], 3)
    q = rand_q(n, heads[0], 128, 60)
    o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints([0, n]), window=window,
                               sinks=sinks, return_lse=True)
    kda.check()
    p = torch.arange(tokens - n, tokens)
    sees = torch.zeros(n, dtype=torch.bool)
    for j in at:
        see = j <= p
        if window:
            see &= (j > p - window) | torch.tensor(j < sinks)
        sees |= see
    x = o[..., 3].float().cpu()
    if which == 0:
        assert x[sees].isnan().all()
    else:
        assert (x[sees] == VALUES[which]).all()
    clean = dict(c, v=torch.nan_to_num(c["v"], 0, 0, 0) if dtype == BF16 else c["v"])
    if dtype == E4M3:
        raw = c["v"].view(torch.uint8).clone()
        raw[raw == 0x7F] = 0
        clean = dict(c, v=raw.view(E4M3))
    ref = ref_prefill(q, clean, [n], 128 ** -0.5, window, sinks)
    other = [d for d in range(128) if d != 3]
    check_attention(o[..., other], lse, [y[..., other] if y.dim() == 3 and y.shape[-1] == 128
                                         else y for y in ref])
    if not sees.all():
        check_attention(*rows_of(o, lse, ref, ~sees))


def test_infinities_of_both_signs_make_nan():
    c = make_cache([300], 32, 1, 64, BF16, 61)
    poisoned(c, 0, 100, math.inf, 3)
    poisoned(c, 0, 250, -math.inf, 3)
    poisoned(c, 0, 130, -math.inf, 40)
    q = rand_q(300, 1, 64, 62)
    o = kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints([0, 300])).float()
    kda.check()
    assert o[:100].isfinite().all()
    assert (o[100:250, 0, 3] == math.inf).all() and o[250:, 0, 3].isnan().all()
    assert o[:130].isfinite()[..., 40].all() and (o[130:, 0, 40] == -math.inf).all()


# ---- refused requests and the tokens that were meant for them ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("packed", [False, True])
def test_tokens_of_a_refused_row_are_dropped(packed, dtype):
    """Rows 0 and 1 share a full page, the pool has one page left, rows 0, 1 and 2
    each need one: row 0 gets it, and the tokens of the others change nothing."""
    page, HKV, D, pages = 16, 1, 64, 5
    k = torch.zeros(pages, page, HKV, D, device="cuda").to(dtype)
    v = k.clone()
    cache, book = kda.KVPages(k, v), kda.PageBook(pages, page, [k, v])
    table = torch.full((5, 4), -1, dtype=torch.int32, device="cuda")
    lens, refs = ints([0] * 5), ints([0] * pages)
    granted = ints([9] * 5)
    args = table, lens, refs

    def tokens(n, value):
        return torch.full((n, HKV, D), value, dtype=BF16, device="cuda")

    book.extend(ints([32, 0, 16, 5, 0]), *args, granted=granted)
    assert granted.tolist() == [32, 0, 16, 5, 0]
    x = tokens(53, 1.0)
    kda.paged_append(cache, x, x, table, lens, ints([0, 32, 32, 48, 53, 53]), granted=granted)
    book.fork(ints([0]), ints([1]), *args)
    kda.check()
    assert lens.tolist() == [32, 32, 16, 5, 0] and int((refs == 0).sum()) == 1
    before = k.clone(), v.clone()
    if packed:
        n = [2, 3, 1, 1, 0]
        book.extend(ints(n), *args, granted=granted)
        x = torch.cat([tokens(m, 2.0 + i) for i, m in enumerate(n)])
        cu = ints([0] + n).cumsum(0).to(torch.int32)
        kda.paged_append(cache, x, x, table, lens, cu, granted=granted)
    else:
        n = [1, 1, 1, 1, 0]
        book.extend(1, *args, granted=granted)
        x = torch.cat([tokens(1, 2.0 + i) for i in range(5)])
        kda.paged_append(cache, x, x, table, lens, granted=granted)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 8
    assert granted.tolist() == [n[0], 0, 0, n[3], 0]
    assert lens.tolist() == [32 + n[0], 32, 16, 5 + n[3], 0]
    for pool, old in zip((k, v), before):
        want = old.clone().float()
        want[table[0, 2].item(), :n[0]] = 2.0
        want[table[3, 0].item(), 5:5 + n[3]] = 5.0
        assert torch.equal(pool.float(), want)


def test_granted_of_requests_that_cannot_be():
    book = kda.PageBook(9, 16)
    table = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    args = table, ints([0, 3, 0, 0]), ints([0] * 9)
    table[1, 0] = 8
    args[2][8] = 1
    granted = ints([7] * 4)
    book.extend(ints([33, -1, 20, 0]), *args, granted=granted)
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2
    assert granted.tolist() == [0, 0, 20, 0] and args[1].tolist() == [0, 3, 20, 0]
    with pytest.raises(kda.KdaError) as e:
        book.extend(1, *args, granted=granted[:3])
    assert e.value.status == 1
    k = torch.zeros(9, 16, 1, 64, dtype=BF16, device="cuda")
    x = torch.ones(4, 1, 64, dtype=BF16, device="cuda")
    with pytest.raises(kda.KdaError) as e:
        kda.paged_append(kda.KVPages(k, k), x, x, table, args[1], granted=granted.long())
    assert e.value.status == 1
    kda.check()


# ---- streams ----

@pytest.mark.parametrize("call", ["decode", "prefill", "extend"])
def test_memory_of_a_call_on_another_stream(call):
    """Memory that was given back on the current stream, where work on it is still
    queued, is not written early by a call on another stream."""
    c = make_cache([100] * 64, 32, 2, 128, BF16, 63, poison=False)
    q, pages = rand_q(64, 32, 128, 64), kv(c)
    ws = kda.paged_decode_workspace(pages, 64, 32)
    side = torch.cuda.Stream()
    cu = torch.arange(65, dtype=torch.int32, device="cuda")
    lse = torch.empty(64, 32, device="cuda")
    table = torch.full((2, 30000), -1, dtype=torch.int32, device="cuda")
    args = table, ints([0, 0]), ints([0] * 40000)
    add = ints([450000, 10])
    def run():
        if call == "decode":
            kda.paged_decode(q, pages, c["table"], c["lens"], lse=lse, workspace=ws, stream=side)
        elif call == "prefill":
            kda.paged_prefill(q, pages, c["table"], c["lens"], cu, lse=lse, stream=side)
        else:
            kda.PageBook(40000, 16).extend(add, *args, stream=side)

    run()                                     # (a first launch may wait for the GPU)
    torch.cuda.synchronize()
    args[1].zero_()
    args[2].zero_()
    need = 1 << 19                            # bytes of q, and about the book's workspace
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # every free piece of that size, all given back with a copy of them still queued
    ys = torch.zeros(256, need, dtype=torch.uint8, device="cuda")
    xs = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    held = torch.cuda.memory_reserved()
    while held == torch.cuda.memory_reserved():
        xs.append(torch.full((need,), 7, dtype=torch.uint8, device="cuda"))
    xs.pop()
    torch.cuda.empty_cache()
    n = len(xs)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    for x, y in zip(xs, ys):
        y.copy_(x)
    del x, xs
    run()
    torch.cuda.synchronize()
    kda.check()
    assert (ys[:n] == 7).all()


# ---- errors ----

def test_one_check_reports_and_clears_every_error():
    c = make_cache([40, 20], 16, 1, 64, BF16, 65, poison=False)
    q = rand_q(2, 2, 64, 66)
    bad = ints([-1, 20])
    for _ in range(2):
        kda.paged_append(kv(c), q[:, :1], q[:, 1:], c["table"] - 5000, c["lens"])
        kda.paged_decode(q, kv(c), c["table"], bad)
        kda.paged_prefill(q, kv(c), c["table"], bad, ints([0, 1, 2]))
        kda.PageBook(4, 16).extend(-1 * ints([1]), ints([[-1]]), ints([0]), ints([0] * 4))
        with pytest.raises(kda.KdaError) as e:
            kda.check()
        assert e.value.status == 2
        kda.check()


# ---- windows and tables ----

@pytest.mark.parametrize("window", [10, 79, 80, 1 << 20, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_windows_as_wide_as_can_be(dtype, window):
    """A window past any length hides nothing, with queries before the first
    token too."""
    lens, qn = [10, 0, 70], [30, 4, 75]
    c = make_cache(lens, 16, 1, 64, dtype, 67)
    c = dict(c, table=c["table"].contiguous())
    q = rand_q(sum(qn), 2, 64, 68)
    cu = ints([0] + qn).cumsum(0).to(torch.int32)
    o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], cu, window=window, sinks=3,
                               return_lse=True)
    d, dl = kda.paged_decode(q[:3], kv(c), c["table"], c["lens"], window=window, sinks=2 ** 31 - 1,
                             return_lse=True)
    kda.check()
    check_attention(o, lse, ref_prefill(q, c, qn, 0.125, window, 3))
    check_attention(d, dl, ref_decode(q[:3], c, 0.125, window, 2 ** 31 - 1))


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_pages_behind_the_window_may_be_released(dtype, sinks, page):
    """A window layer may give pages back that no query sees any more: they are
    not read, and not reported."""
    tokens, n, window = 1000, 20, 300
    c = make_cache([tokens], page, 2, 64, dtype, 69)
    low = tokens - n - window + 1              # the first token that a query sees
    gone = [i for i in range(low // page) if i * page >= sinks]
    keep = c["table"].clone()
    c["table"][0, gone] = -1
    q = rand_q(n, 4, 64, 70)
    for wide in (0, 4096):
        t = widened(c, wide)["table"] if wide else c["table"]
        o, lse = kda.paged_prefill(q, kv(c), t, c["lens"], ints([0, n]), window=window,
                                   sinks=sinks, return_lse=True)
        kda.check()
        check_attention(o, lse, ref_prefill(q, dict(c, table=keep), [n], 0.125, window, sinks))
    d, dl = kda.paged_decode(q[-1:], kv(c), c["table"], c["lens"], window=window, sinks=sinks,
                             return_lse=True)
    kda.check()
    check_attention(d, dl, ref_decode(q[-1:], dict(c, table=keep), 0.125, window, sinks))


# ---- pools with a dimension of one ----

def test_strides_of_a_dimension_of_one_do_not_matter():
    g = torch.Generator().manual_seed(74)
    k = torch.randn(6, 1, 16, 64, generator=g).to(BF16).cuda().transpose(1, 2)
    v = torch.randn(6, 16, 1, 64, generator=g).to(BF16).cuda()
    assert k.shape == v.shape and k.stride() != v.stride()
    table, lens = ints([[3, 1, 5]]), ints([40])
    q = rand_q(1, 4, 64, 75)
    o = kda.paged_decode(q, kda.KVPages(k, v), table, lens)
    same = kda.paged_decode(q, kda.KVPages(k.contiguous(), v), table, lens)
    kda.check()
    assert torch.equal(o, same)


# ---- queries of unequal channels ----

@pytest.mark.parametrize("amp", [2.0 ** 8, 2.0 ** 20, 2.0 ** 27])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("prefill", [False, True])
def test_query_channels_far_larger_than_others(prefill, dtype, amp):
    """One channel of q is far larger than the others and meets keys of zero: the logits
    are the other channels' (their error is bounded by the sum of |q k| alone)."""
    c = make_cache([700], 32, 2, 128, dtype, 78, poison=False)
    k = c["k"].view(torch.uint8) if dtype == E4M3 else c["k"]
    k[..., 17] = 0
    q = rand_q(300 if prefill else 1, 4, 128, 79)
    q[..., 17] = amp
    if prefill:
        o, lse = kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints([0, 300]),
                                   return_lse=True)
        ref = ref_prefill(q, c, [300], 128 ** -0.5)
    else:
        o, lse = kda.paged_decode(q, kv(c), c["table"], c["lens"], return_lse=True)
        ref = ref_decode(q, c, 128 ** -0.5)
    kda.check()
    check_attention(o, lse, ref)


@pytest.mark.parametrize("scale", [0.74, 0.75, 0.7513, 0.752, 0.76, -0.7513])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_neighbouring_logits_whose_products_round_alike(dtype, scale):
    """S of later keys is the next float above that of earlier ones, 2^5 at 2^29, so that
    the logits differ by 30 and more in base 2: later keys alone count where they are
    seen, though scale S may round to the same number.  Bound as above."""
    c = make_cache([600], 32, 1, 128, dtype, 80, poison=False)
    if c["ks"] is not None:
        c["ks"].fill_(1.0)
    c["k"].zero_()
    c["k"][..., 0] = 1.0
    late = 200
    raw = c["k"].view(torch.uint8) if dtype == E4M3 else c["k"]
    one = raw[c["table"][0, 0].item(), 0, 0, 0].item()
    for j in range(late, 600):
        raw[c["table"][0, j // 32].item(), j % 32, 0, 1] = one
    q = torch.zeros(600, 2, 128, dtype=BF16, device="cuda")
    q[..., 0] = math.copysign(1.9375 * 2.0 ** 28, scale)
    q[..., 1] = math.copysign(2.0 ** 5, scale)
    o = kda.paged_prefill(q, kv(c), c["table"], c["lens"], ints([0, 600]), scale=scale)
    kda.check()
    assert o.isfinite().all()
    v = tokens_of(c["v"], c["vs"], c["table"], 0, 600)[:, 0]
    i = torch.arange(1, 601, dtype=torch.float64)[:, None]
    n = torch.where(i > late, i - late, i)
    mean, big = (torch.cat((x[:late].cumsum(0), x[late:].cumsum(0))) / n for x in (v, v.abs()))
    bound = (2.0 ** -8 * mean.abs() + 2.0 ** -10 * big)[:, None]
    assert ((o.double().cpu() - mean[:, None]).abs() <= bound).all()
