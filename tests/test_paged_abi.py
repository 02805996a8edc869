"""The paged cache's C ABI without a GPU: bad arguments are refused before any
launch, and empty calls succeed without one."""
import ctypes

import pytest

from gated_delta_rule_41_gb300 import build as kbuild
from gated_delta_rule_41_gb300 import paged
from gated_delta_rule_41_gb300.paged import KdaPagedDims, KdaPagePool, KdaPagesDims

FAKE, ODD = 1 << 20, (1 << 20) + 1      # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return paged._lib()


def dims(**kw):
    base = dict(S=2, HQ=8, HKV=2, D=128, num_pages=10, page_size=16, max_pages=4, cache_dtype=1,
                page_stride=16 * 256, token_stride=256, head_stride=128, scale=0.1, window=0,
                sinks=0)
    base.update(kw)
    return KdaPagedDims(**base)


def decode(lib, d, q=FAKE, q_stride=1024, kp=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=None,
           ws=FAKE, n=1 << 30):
    return lib.kda_paged_decode(d, q, q_stride, kp, FAKE, None, None, table, lens, o, lse, ws, n,
                                None)


def prefill(lib, d, T=5, cu=FAKE, q=FAKE, q_stride=1024, ws=FAKE, n=1 << 30):
    return lib.kda_paged_prefill(d, cu, T, q, q_stride, FAKE, FAKE, None, None, FAKE, FAKE, FAKE,
                                 None, ws, n, None)


def append(lib, d, T=2, cu=None, k=FAKE, stride=256, kp=FAKE):
    return lib.kda_paged_append(d, cu, T, k, stride, FAKE, stride, None, None, FAKE, FAKE, kp,
                                FAKE, None)


BAD = [(dict(S=-1), 2), (dict(HKV=0), 2), (dict(num_pages=0), 2), (dict(max_pages=0), 2),
       (dict(D=96), 3), (dict(page_size=24), 3), (dict(page_size=8), 3), (dict(page_size=512), 3),
       (dict(cache_dtype=0), 3), (dict(cache_dtype=5), 1), (dict(S=70000), 3),
       (dict(max_pages=1 << 27), 3), (dict(token_stride=4), 4), (dict(head_stride=-128), 2),
       (dict(cache_dtype=2, token_stride=8), 4), (dict(num_pages=(1 << 30) + 1), 3)]
BAD_ATTEND = [(dict(HQ=9), 2), (dict(HQ=130), 3), (dict(window=-1), 1), (dict(sinks=-2), 1),
              (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1)]


@pytest.mark.parametrize("kw,want", BAD)
def test_dims_refused_everywhere(lib, kw, want):
    d = dims(**kw)
    assert decode(lib, d) == want and prefill(lib, d) == want and append(lib, d) == want
    assert lib.kda_paged_decode_workspace_bytes(d) == 0
    assert lib.kda_paged_prefill_workspace_bytes(d, 5) == 0


@pytest.mark.parametrize("kw,want", BAD_ATTEND)
def test_attention_dims_refused(lib, kw, want):
    assert decode(lib, dims(**kw)) == want and prefill(lib, dims(**kw)) == want


def test_pointers(lib):
    d = dims()
    assert lib.kda_paged_decode(None, *([FAKE, 8] + [FAKE] * 9 + [0, None])) == 1
    for name in ("q", "kp", "table", "lens", "o"):
        assert decode(lib, d, **{name: None}) == 1
        assert decode(lib, d, **{name: ODD}) == 4
    assert decode(lib, d, lse=ODD) == 4
    assert decode(lib, d, q_stride=1020) == 2 and decode(lib, d, q_stride=1028) == 4
    need = lib.kda_paged_decode_workspace_bytes(d)
    if need:
        assert decode(lib, d, ws=None) == 5 and decode(lib, d, n=need - 1) == 5
        assert decode(lib, d, ws=FAKE + 16) == 4
    assert prefill(lib, d, cu=None) == 1 and prefill(lib, d, cu=ODD) == 4
    assert prefill(lib, d, T=-1) == 2 and prefill(lib, d, T=1 << 28) == 3
    assert prefill(lib, d, q=FAKE + 8) == 4
    need = lib.kda_paged_prefill_workspace_bytes(d, 5)
    if need:
        assert prefill(lib, d, ws=None) == 5 and prefill(lib, d, n=need - 1) == 5
    assert append(lib, d, T=3) == 2                    # one token each: T == S
    assert append(lib, d, k=None) == 1 and append(lib, d, k=ODD) == 4
    assert append(lib, d, stride=128) == 2 and append(lib, d, stride=260) == 4
    assert append(lib, d, cu=ODD) == 4


def test_empty_calls(lib):
    assert decode(lib, dims(S=0)) == 0
    assert prefill(lib, dims(), T=0) == 0 and prefill(lib, dims(S=0), T=3) == 2
    assert append(lib, dims(), T=0, cu=FAKE) == 0


def pool(base=FAKE, stride=4096, page=4096):
    return (KdaPagePool * 1)(KdaPagePool(base, stride, page))


def test_bookkeeping(lib):
    g = KdaPagesDims(4, 8, 100, 16)
    need = lib.kda_pages_workspace_bytes(g)
    assert need > 0 and need % 256 == 0
    for bad, want in ((KdaPagesDims(-1, 8, 100, 16), 2), (KdaPagesDims(4, 0, 100, 16), 2),
                      (KdaPagesDims(4, 8, 0, 16), 2), (KdaPagesDims(4, 8, 100, 0), 2),
                      (KdaPagesDims(70000, 8, 100, 16), 3),
                      (KdaPagesDims(4, 8, (1 << 30) + 1, 16), 3),
                      (KdaPagesDims(4, 1 << 27, 100, 16), 3)):
        assert lib.kda_pages_workspace_bytes(bad) == 0
        assert lib.kda_pages_extend(bad, None, 1, FAKE, FAKE, FAKE, FAKE, need, None) == want
        assert lib.kda_pages_free(bad, FAKE, 1, FAKE, FAKE, FAKE, None) == want

    def fork(p=None, np=1, n=2, parents=FAKE, ws=FAKE, size=need):
        return lib.kda_pages_fork(g, p if p is not None else pool(), np, parents, FAKE, n, FAKE,
                                  FAKE, FAKE, ws, size, None)

    assert fork(n=5) == 2 and fork(n=-1) == 2 and fork(parents=None) == 1
    assert fork(parents=ODD) == 4 and fork(ws=None) == 5 and fork(size=need - 1) == 5
    assert fork(ws=FAKE + 4) == 4 and fork(np=65) == 3 and fork(np=-1) == 2
    assert fork(p=pool(base=None)) == 1 and fork(p=pool(base=FAKE + 8)) == 4
    assert fork(p=pool(page=8192)) == 2 and fork(p=pool(page=4088)) == 4
    assert fork(n=0) == 0
    assert lib.kda_pages_extend(g, None, -1, FAKE, FAKE, FAKE, FAKE, need, None) == 2
    assert lib.kda_pages_extend(g, None, 1, None, FAKE, FAKE, FAKE, need, None) == 1
    assert lib.kda_pages_free(g, None, 1, FAKE, FAKE, FAKE, None) == 1
    assert lib.kda_pages_free(g, FAKE, 0, FAKE, FAKE, FAKE, None) == 0
    assert lib.kda_pages_compact(g, pool(), 1, FAKE, None, FAKE, need, None) == 1
    assert lib.kda_pages_compact(g, pool(), 1, FAKE, FAKE, None, 0, None) == 5
    assert lib.kda_pages_copy(pool(), 1, 0, FAKE, FAKE, 3, None) == 2
    assert lib.kda_pages_copy(pool(), 1, 10, None, FAKE, 3, None) == 1
    assert lib.kda_pages_copy(pool(), 1, 10, FAKE, FAKE, 0, None) == 0


def test_status_string(lib):
    lib.kda_status_str.restype = ctypes.c_char_p
    assert lib.kda_status_str(8) == b"too few free pages"
