"""Paged key-value cache at its edges: refused calls, values and logits that
are not ordinary numbers, tables with released pages, streams and errors."""
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
