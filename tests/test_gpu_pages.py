"""Page bookkeeping on the GPU against host lists (tables, lengths, counts and
pool contents, all exact), and a serving loop that uses everything together."""
import random

import pytest
import torch

import gated_delta_rule_41_gb300 as kda
from paged_util import Book, check_attention, ref_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_41_gb300 import build
    build.build()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def start(S, width, pages, page, n_pools=2, seed=0, row=32):
    g = torch.Generator().manual_seed(seed)
    pools = [torch.randint(0, 1 << 15, (pages, page, row), generator=g, dtype=torch.int32)
             for _ in range(n_pools)]
    table = torch.full((S, width), -1, dtype=torch.int32)
    lens, refs = torch.zeros(S, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32)
    host = Book(table, lens, refs, page, pools)
    dev = [table.cuda(), lens.cuda(), refs.cuda()]
    dpools = [p.cuda() for p in pools]
    return host, dev, dpools, kda.PageBook(pages, page, dpools)


def same(host, dev, dpools):
    assert dev[0].tolist() == host.table
    assert dev[1].tolist() == host.lens
    assert dev[2].tolist() == host.refs
    for a, b in zip(dpools, host.pools):
        assert torch.equal(a.cpu(), b)


def check(host):
    if host.refused:
        with pytest.raises(kda.KdaError) as e:
            kda.check()
        assert e.value.status == 8
        host.refused = False
    else:
        kda.check()


@pytest.mark.parametrize("S,width,pages,page", [(1, 1, 1, 16), (7, 9, 40, 16), (40, 30, 500, 16),
                                                (300, 20, 9000, 64), (2000, 5, 5003, 7)])
def test_random_sequences_of_calls(S, width, pages, page):
    """Prompts come, grow, fork and go, with the pool running short at times."""
    rng = random.Random(S)
    host, dev, dpools, book = start(S, width, pages, page, row=4 if pages > 1000 else 32)
    for step in range(25):
        live = [s for s in range(S) if host.lens[s] > 0]
        idle = [s for s in range(S) if host.lens[s] == 0]
        op = rng.choice(["prompt", "prompt", "grow", "fork", "free", "compact"])
        if op == "prompt":
            add = [0] * S
            for s in rng.sample(idle, min(len(idle), rng.randint(1, 1 + S // 4))):
                add[s] = rng.randint(0, width * page)
            book.extend(ints(add), *dev)
            host.extend(add)
        elif op == "grow":
            if any(n + 1 > width * page for n in host.lens):
                continue
            book.extend(1, *dev)
            host.extend([int(n > 0) for n in host.lens])
        elif op == "fork" and live and idle:
            n = rng.randint(1, len(idle))
            par = [rng.choice(live) for _ in range(n)]
            ch = rng.sample(idle, n)
            book.fork(ints(par), ints(ch), *dev)
            host.fork(par, ch)
        elif op == "free" and live:
            slots = rng.sample(live, rng.randint(1, len(live)))
            book.free(ints(slots), *dev)
            host.free(slots)
        elif op == "compact":
            book.compact(*dev)
            host.compact()
        check(host)
        same(host, dev, dpools)


def test_extend_refuses_whole_requests_in_order():
    host, dev, dpools, book = start(4, 8, 10, 16)
    add = [33, 100, 40, 0]            # 3 + 7 pages, then 3 more that are not there
    book.extend(ints(add), *dev)
    host.extend(add)
    assert host.refused and host.lens == [33, 100, 0, 0]
    check(host)
    same(host, dev, dpools)
    book.extend(1, *dev)              # 34 and 101 need no page
    host.extend([1, 1, 0, 0])
    check(host)
    same(host, dev, dpools)


def test_fork_refused_child_stays_idle():
    host, dev, dpools, book = start(6, 4, 4, 16)
    add = [20, 0, 0, 0, 0, 0]
    book.extend(ints(add), *dev)
    host.extend(add)
    par, ch = [0, 0, 0], [2, 3, 4]
    book.fork(ints(par), ints(ch), *dev)
    host.fork(par, ch)
    assert host.refused and host.lens == [20, 0, 20, 20, 0, 0]
    check(host)
    same(host, dev, dpools)


def test_bad_rows_are_reported_and_skipped():
    host, dev, dpools, book = start(4, 4, 20, 16)
    add = [20, 5, 0, 0]
    book.extend(ints(add), *dev)
    host.extend(add)
    kda.check()
    for call in (lambda: book.extend(ints([0, -1, 0, 0]), *dev),
                 lambda: book.extend(ints([0, 0, 65, 0]), *dev),
                 lambda: book.fork(ints([0]), ints([1]), *dev),       # the child is not idle
                 lambda: book.fork(ints([9]), ints([2]), *dev),
                 lambda: book.fork(ints([0]), ints([-1]), *dev),
                 lambda: book.free(ints([4]), *dev)):
        call()
        with pytest.raises(kda.KdaError) as e:
            kda.check()
        assert e.value.status == 2
        same(host, dev, dpools)
    book.fork(ints([3]), ints([2]), *dev)      # an idle parent: an idle child
    kda.check()
    same(host, dev, dpools)


def test_pages_copy_pools_of_any_page_size_and_stride():
    """Recurrent states (one block per slot) and page views of a wider pool."""
    g = torch.Generator().manual_seed(3)
    state = torch.randn(9, 4, 128, 128, generator=g).cuda()
    joint = torch.randn(9, 2, 16, 3, 64, generator=g).to(torch.bfloat16).cuda()
    odd = torch.randint(0, 255, (9, 48), generator=g, dtype=torch.uint8).cuda()
    pools = [state, joint[:, 0], joint[:, 1].transpose(1, 2), odd]
    want = [p.clone() for p in pools]
    src, dst = [0, 0, 5, -1, 2], [1, 3, 4, 6, -1]
    for w in want:
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                w[b] = w[a]
    kda.pages_copy(pools, ints(src), ints(dst))
    kda.check()
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    kda.pages_copy(pools, ints([0, 9]), ints([1, 2]))
    with pytest.raises(kda.KdaError) as e:
        kda.check()
    assert e.value.status == 2
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def test_bookkeeping_refusals():
    def status(fn):
        with pytest.raises(kda.KdaError) as e:
            fn()
        return e.value.status

    pool = torch.zeros(8, 16, 64, device="cuda")
    assert status(lambda: kda.PageBook(9, 16, [pool])) == 1
    assert status(lambda: kda.PageBook(8, 16, [pool[:, :, :7]])) == 1
    assert status(lambda: kda.PageBook(8, 16, [pool] * 65)) == 3
    host, dev, dpools, book = start(3, 2, 8, 16)
    assert status(lambda: book.fork(ints([0]), ints([1, 2]), *dev)) == 1
    assert status(lambda: book.fork(ints([0] * 4), ints([1] * 4), *dev)) == 2
    assert status(lambda: book.extend(-1, *dev)) == 2
    assert status(lambda: book.extend(1, dev[0].long(), dev[1], dev[2])) == 1
    assert status(lambda: book.free(ints([0]), dev[0], dev[1], dev[2][:4])) == 1
    odd = torch.zeros(8, 5, dtype=torch.uint8, device="cuda")
    assert status(lambda: kda.pages_copy([odd], ints([0]), ints([1]))) == 4


def test_serving_loop():
    """Prompts, decode steps, a fork, released rows and a compaction; after each
    step the attention over the pages equals the reference over the tokens that
    each sequence has seen, kept apart in dense lists."""
    S, page, HQ, HKV, D, pages = 6, 16, 4, 2, 64, 40
    g = torch.Generator().manual_seed(5)
    k = torch.full((pages, page, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    cache = kda.KVPages(k, v)
    book = kda.PageBook(pages, page, [k, v])
    table = torch.full((S, 8), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    seen = [torch.zeros(0, 2, HKV, D, dtype=torch.bfloat16) for _ in range(S)]

    def new(n):
        return torch.randn(n, 2, HKV, D, generator=g).to(torch.bfloat16)

    def attend(only):
        q = torch.randn(S, HQ, D, generator=g).to(torch.bfloat16).cuda()
        o, lse = kda.paged_decode(q, cache, table, lens, return_lse=True)
        kda.check()
        most = max(max(len(x) for x in seen), 1)
        dense = torch.zeros(S, most, 2, HKV, D, dtype=torch.bfloat16)
        for s, x in enumerate(seen):
            dense[s, :len(x)] = x
        ref = dict(k=dense[:, :, 0], v=dense[:, :, 1], ks=None, vs=None,
                   table=torch.arange(S, dtype=torch.int32)[:, None],
                   lens=torch.tensor([len(x) for x in seen]))
        assert lens.tolist() == [len(x) for x in seen]
        check_attention(o, lse, ref_decode(q, ref, D ** -0.5))

    def prompts(n):
        xs = [new(m) for m in n]
        book.extend(ints(n), table, lens, refs)
        x = torch.cat(xs).cuda()
        cu = ints([0] + n).cumsum(0).to(torch.int32)
        kda.paged_append(cache, x[:, 0], x[:, 1], table, lens, cu)
        for s, y in enumerate(xs):
            seen[s] = torch.cat((seen[s], y))

    def step():
        book.extend(1, table, lens, refs)
        x = new(S).cuda()
        kda.paged_append(cache, x[:, 0], x[:, 1], table, lens)
        for s in range(S):
            if len(seen[s]):
                seen[s] = torch.cat((seen[s], x[s:s + 1].cpu()))

    prompts([20, 33, 5, 0, 0, 0])
    attend(None)
    for _ in range(14):
        step()
    attend(None)
    book.fork(ints([1, 0]), ints([4, 3]), table, lens, refs)
    seen[4], seen[3] = seen[1], seen[0]
    step()
    attend(None)
    book.free(ints([1]), table, lens, refs)
    seen[1] = seen[1][:0]
    book.compact(table, lens, refs)
    attend(None)
    held = int((refs > 0).sum())
    assert (refs[:held] > 0).all()
    prompts([0, 50, 0, 0, 0, 7])
    step()
    attend(None)


def test_pools_of_many_pages():
    """More pages than one round of the plans' scans, held ones far apart."""
    S, width, pages, page = 500, 40, 50021, 16
    host, dev, dpools, book = start(S, width, pages, page, n_pools=1, row=4)
    rng = random.Random(9)
    add = [rng.randint(0, width * page) for _ in range(S)]
    for step in range(4):
        book.extend(ints(add), *dev)
        host.extend(add)
        check(host)
        same(host, dev, dpools)
        gone = rng.sample(range(S), 300) if step < 3 else list(range(0, S, 2))
        gone = [s for s in gone if host.lens[s]]
        book.free(ints(gone), *dev)
        host.free(gone)
        idle = [s for s in range(S) if host.lens[s] == 0]
        live = [s for s in range(S) if host.lens[s] > 0]
        par, ch = [rng.choice(live) for _ in range(50)], rng.sample(idle, 50)
        book.fork(ints(par), ints(ch), *dev)
        host.fork(par, ch)
        check(host)
        same(host, dev, dpools)
        add = [rng.randint(0, width * page) if host.lens[s] == 0 else 0 for s in range(S)]
    book.compact(*dev)
    host.compact()
    check(host)
    same(host, dev, dpools)


def test_plans_read_counts_at_any_alignment():
    for shift in range(4):
        host, _, dpools, book = start(6, 5, 70, 16)
        buf = torch.zeros(80, dtype=torch.int32, device="cuda")
        dev = [torch.full((6, 5), -1, dtype=torch.int32, device="cuda"),
               torch.zeros(6, dtype=torch.int32, device="cuda"), buf[shift:shift + 70]]
        add = [40, 0, 70, 16, 1, 0]
        book.extend(ints(add), *dev)
        host.extend(add)
        book.free(ints([2]), *dev)
        host.free([2])
        book.fork(ints([0]), ints([5]), *dev)
        host.fork([0], [5])
        book.compact(*dev)
        host.compact()
        kda.check()
        same(host, dev, dpools)
        assert (buf[70 + shift:] == 0).all() and (buf[:shift] == 0).all()
