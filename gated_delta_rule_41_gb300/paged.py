"""Thin ctypes binding of the paged key-value cache of libkda.so (C ABI in
include/kda.h): appending tokens, attention over the pages, page bookkeeping.

A serving loop holds the pools, one block table and one length per sequence,
all on the device:

    pages = KVPages(k, v)                   # pools [num_pages, page_size, HKV, D]
    book = PageBook(num_pages, page_size, pools)
    book.extend(add, table, lens, refs, granted=granted)   # room for the new tokens
    paged_append(pages, k_new, v_new, table, lens, cu_seqlens, granted=granted)
    o = paged_prefill(q, pages, table, lens, cu_seqlens)      # prompts
    o = paged_decode(q, pages, table, lens)                   # one new token each

As in ``kda.py`` every step runs in the library's kernels on the caller's
stream; nothing here waits for the GPU.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import kda as _kda
from .kda import KDA_BF16, KDA_F32, KdaError, _raise

KDA_E4M3 = 2
MAX_POOLS = 64


class KdaPagedDims(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int), ("HQ", ctypes.c_int), ("HKV", ctypes.c_int),
                ("D", ctypes.c_int), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("cache_dtype", ctypes.c_int),
                ("page_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("scale", ctypes.c_float),
                ("window", ctypes.c_int), ("sinks", ctypes.c_int)]


class KdaPagePool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_stride_bytes", ctypes.c_longlong),
                ("page_bytes", ctypes.c_longlong)]


class KdaPagesDims(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = _kda.load_library()
        P, I, L, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
        D, G, O = (ctypes.POINTER(x) for x in (KdaPagedDims, KdaPagesDims, KdaPagePool))
        for name, res, args in (
                ("kda_paged_append", I, [D, P, I, P, L, P, L, P, P, P, P, P, P, P]),
                ("kda_paged_append_granted", I, [D, P, I, P, L, P, L, P, P, P, P, P, P, P, P]),
                ("kda_paged_decode_workspace_bytes", S, [D]),
                ("kda_paged_decode", I, [D, P, L] + [P] * 9 + [S, P]),
                ("kda_paged_prefill_workspace_bytes", S, [D, I]),
                ("kda_paged_prefill", I, [D, P, I, P, L] + [P] * 9 + [S, P]),
                ("kda_pages_workspace_bytes", S, [G]),
                ("kda_pages_fork", I, [G, O, I, P, P, I, P, P, P, P, S, P]),
                ("kda_pages_extend", I, [G, P, I, P, P, P, P, S, P]),
                ("kda_pages_extend_granted", I, [G, P, I, P, P, P, P, P, S, P]),
                ("kda_pages_free", I, [G, P, I, P, P, P, P]),
                ("kda_pages_compact", I, [G, O, I, P, P, P, S, P]),
                ("kda_pages_copy", I, [O, I, I, P, P, I, P])):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _bound = lib
    return _bound


# The current stream's handle, without the Stream object that torch.cuda's
# own call makes for it (a few microseconds of a small call).
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _get_device is None or _get_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _get_stream(_get_device())


def _fresh(stream, shape, dtype, device):
    """A tensor that a launch on ``stream`` writes and the caller goes on with: of
    that stream's memory, since what was given back on the current one may still
    be in use there; and not given back before the current stream is done too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _ints(name, t, dim, n=None):
    if (t.dtype != torch.int32 or not t.is_cuda or t.dim() != dim or not t.is_contiguous()
            or (n is not None and t.shape[0] != n)):
        raise KdaError(1, f"{name} must be a contiguous {dim}-D int32 CUDA tensor"
                          + (f" of {n} rows" if n is not None else ""))
    return t.data_ptr()


def _tokens(name, t, heads, D):
    """A bf16 tensor [T, heads, D] whose tokens may lie apart (a slice of a
    wider projection): its token stride in elements."""
    if t.dtype != torch.bfloat16:
        raise KdaError(3, f"{name}: {t.dtype} (bf16 only)")
    if not t.is_cuda or t.dim() != 3 or t.shape[2] != D or (heads and t.shape[1] != heads):
        raise KdaError(1, f"{name} must be a CUDA tensor [tokens, {heads or 'heads'}, {D}]")
    n, h, _ = t.shape
    a, b, c = t.stride()
    if c != 1 or (h > 1 and b != D):
        raise KdaError(1, f"{name}: the heads of a token must be contiguous")
    return a if n > 1 else h * D


class KVPages:
    """The K and V pools of one attention layer: tensors [num_pages, page_size,
    HKV, D], bf16 or float8_e4m3fn, views of any page, row and head stride with
    contiguous D (a pool kept as [num_pages, HKV, page_size, D] is passed
    transposed).  ``k_scale``, ``v_scale``: float32 [HKV], what an e4m3 code of
    that head is worth (None: 1)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        for n, t in (("k", k), ("v", v)):
            if not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
                raise KdaError(1, f"{n} pool must be a CUDA tensor [pages, rows, HKV, D] with "
                                  "contiguous D")
        # of a dimension of one, torch may report any stride
        st, sv = ([0 if n == 1 else x for n, x in zip(t.shape, t.stride())] for t in (k, v))
        if k.shape != v.shape or k.dtype != v.dtype or st != sv:
            raise KdaError(1, "the K and V pools must share shape, type and strides")
        codes = {torch.bfloat16: KDA_BF16, torch.float8_e4m3fn: KDA_E4M3, torch.float32: KDA_F32}
        if k.dtype not in codes:
            raise KdaError(3, f"cache type {k.dtype} (bf16 or float8_e4m3fn)")
        for n, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is None:
                continue
            if k.dtype != torch.float8_e4m3fn:
                raise KdaError(1, f"{n}: a bf16 cache has no scales")
            if s.dtype != torch.float32 or not s.is_cuda or s.shape != (k.shape[2],) \
                    or not s.is_contiguous():
                raise KdaError(1, f"{n} must be a contiguous float32 CUDA tensor [HKV]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.page_size, self.HKV, self.D = k.shape
        self._code = codes[k.dtype]
        self._strides = tuple(st)
        self._calls = {}   # dims (and workspace bytes) of the calls seen
        self._ptrs = (k.data_ptr(), v.data_ptr(),
                      None if k_scale is None else k_scale.data_ptr(),
                      None if v_scale is None else v_scale.data_ptr())

    def dims(self, S, HQ, max_pages, scale=None, window=0, sinks=0) -> KdaPagedDims:
        st = self._strides
        return KdaPagedDims(S, HQ, self.HKV, self.D, self.num_pages, self.page_size, max_pages,
                            self._code, st[0], st[1], st[2],
                            self.D ** -0.5 if scale is None else scale, window, sinks)


    def _call(self, S, HQ, max_pages, scale, window, sinks, T=None):
        """Dims pointer and workspace bytes of a call, built once per set of
        sizes.  T None: decode; 0: append; else prompt attention of T tokens."""
        key = (S, HQ, max_pages, scale, window, sinks, T)
        got = self._calls.get(key)
        if got is None:
            if len(self._calls) >= 256:
                self._calls.clear()
            d = ctypes.pointer(self.dims(S, HQ, max_pages, scale, window, sinks))
            need = 0
            if T is None:
                need = int(_lib().kda_paged_decode_workspace_bytes(d))
            elif T > 0:
                need = int(_lib().kda_paged_prefill_workspace_bytes(d, T))
            got = self._calls[key] = (d, need)
        return got


def paged_append(pages: KVPages, k, v, block_table, kv_lens, cu_seqlens=None, stream=None,
                 granted=None):
    """Write new tokens k, v [T, HKV, D] (bf16; slices of a wider projection
    will do) into the pages.  ``kv_lens`` [S] counts the new tokens already:
    with ``cu_seqlens`` [S + 1] sequence s owns tokens cu_seqlens[s] to
    cu_seqlens[s + 1] and they become its last ones; without, one each.
    ``granted`` [S], from ``PageBook.extend``: tokens of a row that gained none
    are dropped; without it they would replace the last ones of a refused row."""
    lib = _lib()
    ks, vs = _tokens("k", k, pages.HKV, pages.D), _tokens("v", v, pages.HKV, pages.D)
    T, (S, width) = k.shape[0], block_table.shape
    if v.shape[0] != T:
        raise KdaError(2, "paged_append: k and v differ in tokens")
    table, lens = _ints("block_table", block_table, 2), _ints("kv_lens", kv_lens, 1, S)
    cu = None if cu_seqlens is None else _ints("cu_seqlens", cu_seqlens, 1, S + 1)
    d, _ = pages._call(S, pages.HKV, width, None, 0, 0, 0)
    kp, vp, sk, sv = pages._ptrs
    got = None if granted is None else _ints("granted", granted, 1, S)
    _raise(lib.kda_paged_append_granted(d, cu, T, k.data_ptr(), ks, v.data_ptr(), vs, sk, sv, table,
                                        lens, got, kp, vp, _raw_stream(stream)),
           "kda_paged_append")


def _attention_workspace(need, workspace, device, stream):
    if need == 0:
        return None
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        return workspace
    # zeroed on the launch's stream: the joining CTAs count from zero
    with torch.cuda.stream(stream):
        return torch.zeros(need, dtype=torch.uint8, device=device)


def _outputs(q, out, lse, return_lse, stream):
    if out is None:
        out = _fresh(stream, q.shape, q.dtype, q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_cuda \
            or not out.is_contiguous():
        raise KdaError(1, "out must be a contiguous CUDA tensor of q's shape and type")
    if lse is None:
        if return_lse:
            lse = _fresh(stream, q.shape[:2], torch.float32, q.device)
    elif lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_cuda \
            or not lse.is_contiguous():
        raise KdaError(1, "lse must be a contiguous float32 CUDA tensor [rows, HQ]")
    return out, lse


def paged_decode_workspace(pages: KVPages, S, HQ, max_pages=1) -> Optional[torch.Tensor]:
    """A workspace for ``paged_decode`` calls of S sequences and HQ heads (any
    lengths), zeroed as it must be before its first use.  Calls that overlap on
    the GPU need one each.  (A call that gets none, or a smaller one, makes a
    fresh one for itself.)"""
    need = int(_lib().kda_paged_decode_workspace_bytes(pages.dims(S, HQ, max_pages)))
    return torch.zeros(need, dtype=torch.uint8, device=pages.k.device) if need else None


def paged_decode(q, pages: KVPages, block_table, kv_lens, scale=None, window=0, sinks=0, out=None,
                 lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of one new token per sequence: q [S, HQ, D] -> o [S, HQ, D]
    (and lse [S, HQ] with ``return_lse``).  The token's own key and value are in
    the cache and counted in ``kv_lens``.  A sequence without tokens gets zeros
    (lse -inf)."""
    lib = _lib()
    qs = _tokens("q", q, 0, pages.D)
    S, HQ, _ = q.shape
    if block_table.shape[0] != S:
        raise KdaError(2, "paged_decode: block_table has other rows than q")
    table, lens = _ints("block_table", block_table, 2), _ints("kv_lens", kv_lens, 1, S)
    d, need = pages._call(S, HQ, block_table.shape[1], scale, window, sinks)
    out, lse = _outputs(q, out, lse, return_lse, stream)
    ws = _attention_workspace(need, workspace, q.device, stream)
    kp, vp, sk, sv = pages._ptrs
    _raise(lib.kda_paged_decode(d, q.data_ptr(), qs, kp, vp, sk, sv, table, lens, out.data_ptr(),
                                None if lse is None else lse.data_ptr(),
                                None if ws is None else ws.data_ptr(), need,
                                _raw_stream(stream)), "kda_paged_decode")
    return (out, lse) if return_lse else out


def paged_prefill_workspace(pages: KVPages, S, T, HQ, max_pages=1) -> Optional[torch.Tensor]:
    """A workspace for ``paged_prefill`` calls of T query tokens in S sequences.
    (What they need does not rise with T throughout; a call that gets none, or a
    smaller one, makes a fresh one for itself.)"""
    need = int(_lib().kda_paged_prefill_workspace_bytes(pages.dims(S, HQ, max_pages), T))
    return torch.zeros(need, dtype=torch.uint8, device=pages.k.device) if need else None


def paged_prefill(q, pages: KVPages, block_table, kv_lens, cu_seqlens, scale=None, window=0,
                  sinks=0, out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Causal attention of prompt tokens q [T, HQ, D], packed: sequence s owns
    tokens cu_seqlens[s] to cu_seqlens[s + 1], the last ones of its
    ``kv_lens[s]`` tokens in the cache (a prompt may come in chunks).  Returns
    o [T, HQ, D], and lse [T, HQ] with ``return_lse``."""
    lib = _lib()
    qs = _tokens("q", q, 0, pages.D)
    T, HQ, _ = q.shape
    S, width = block_table.shape
    table, lens = _ints("block_table", block_table, 2), _ints("kv_lens", kv_lens, 1, S)
    cu = _ints("cu_seqlens", cu_seqlens, 1, S + 1)
    d, need = pages._call(S, HQ, width, scale, window, sinks, T)
    out, lse = _outputs(q, out, lse, return_lse, stream)
    ws = _attention_workspace(need, workspace, q.device, stream)
    kp, vp, sk, sv = pages._ptrs
    _raise(lib.kda_paged_prefill(d, cu, T, q.data_ptr(), qs, kp, vp, sk, sv, table, lens,
                                 out.data_ptr(), None if lse is None else lse.data_ptr(),
                                 None if ws is None else ws.data_ptr(), need,
                                 _raw_stream(stream)), "kda_paged_prefill")
    return (out, lse) if return_lse else out


def _pool_array(pools, num_pages):
    arr = (KdaPagePool * max(1, len(pools)))()
    for i, t in enumerate(pools):
        if not t.is_cuda or t.dim() < 2 or t.shape[0] != num_pages:
            raise KdaError(1, f"pool {i} must be a CUDA tensor [num_pages, ...]")
        # one page is one run of bytes, in whatever order of its dimensions
        run = 1
        for n, st in sorted(zip(t.shape[1:], t.stride()[1:]), key=lambda x: x[1]):
            if n > 1 and st != run:
                raise KdaError(1, f"pool {i}: a page must be contiguous")
            run *= n
        e = t.element_size()
        stride = t.stride(0) if num_pages > 1 else run
        arr[i] = KdaPagePool(t.data_ptr(), stride * e, run * e)
    return arr


def pages_copy(pools: Sequence[torch.Tensor], src, dst, stream=None):
    """Copy page src[i] to page dst[i] of every pool [num_pages, ...]; pairs
    with a negative id are skipped.  No page may be written twice, or be both
    read and written.  Pools of one block per sequence work too: recurrent
    states [slots, HV, K, V] follow a fork with src = parents, dst = children."""
    if not pools:
        return
    n, N = src.shape[0], pools[0].shape[0]
    a, b = _ints("src", src, 1), _ints("dst", dst, 1, n)
    _raise(_lib().kda_pages_copy(_pool_array(pools, N), len(pools), N, a, b, n,
                                 _raw_stream(stream)), "kda_pages_copy")


class PageBook:
    """Page bookkeeping for pools [num_pages, ...] that share their page ids
    (the K and V pools of every layer).  The tables are the caller's device
    tensors, updated in place in stream order: block_table int32 [S, max_pages]
    (-1: no page), kv_lens int32 [S], refs int32 [num_pages] (0: free).  Pages
    are taken lowest id first.  Refused requests (too few free pages) show in
    ``check()`` as KdaError with status 8; their rows stay as they were, and the
    new tokens meant for them are dropped if ``extend``'s ``granted`` goes on to
    ``paged_append``.

    A PageBook keeps one workspace: its calls belong on one stream at a time."""

    def __init__(self, num_pages, page_size, pools: Sequence[torch.Tensor] = ()):
        self.num_pages, self.page_size, self.pools = num_pages, page_size, list(pools)
        if len(self.pools) > MAX_POOLS:
            raise KdaError(3, f"{len(self.pools)} pools (at most {MAX_POOLS})")
        self._arr = _pool_array(self.pools, num_pages)
        self._ws, self._need, self._home, self._dims = None, 0, None, {}

    def _args(self, block_table, kv_lens, refs, stream):
        table = _ints("block_table", block_table, 2)
        S, width = block_table.shape
        lens = _ints("kv_lens", kv_lens, 1, S)
        counts = _ints("refs", refs, 1, self.num_pages)
        got = self._dims.get((S, width))
        if got is None:
            if len(self._dims) >= 256:
                self._dims.clear()
            d = ctypes.pointer(KdaPagesDims(S, width, self.num_pages, self.page_size))
            got = self._dims[S, width] = (d, int(_lib().kda_pages_workspace_bytes(d)))
        d, need = got
        if need > self._need:
            self._ws = _fresh(stream, need, torch.uint8, refs.device)
            self._need, self._home = need, _raw_stream(stream)
        elif self._ws is not None and _raw_stream(stream) != self._home:
            # not given back before that one is done
            self._ws.record_stream(torch.cuda.current_stream() if stream is None else stream)
        return (d, table, lens, counts, None if self._ws is None else self._ws.data_ptr(),
                self._need)

    def fork(self, parents, children, block_table, kv_lens, refs, stream=None):
        """Rows ``children`` (idle ones) become copies of rows ``parents``: full
        pages are shared, the partial last page is copied in every pool."""
        d, table, lens, counts, ws, n_ws = self._args(block_table, kv_lens, refs, stream)
        n = parents.shape[0]
        p, c = _ints("parents", parents, 1), _ints("children", children, 1, n)
        _raise(_lib().kda_pages_fork(d, self._arr, len(self.pools), p, c, n, table, lens, counts,
                                     ws, n_ws, _raw_stream(stream)), "kda_pages_fork")

    def extend(self, add, block_table, kv_lens, refs, stream=None, granted=None):
        """Lengths grow by ``add`` (int32 [S]; or an int, for the rows with
        tokens), and rows get the pages they then need.  ``granted`` (int32 [S],
        written): the tokens that each row gained, for ``paged_append``."""
        d, table, lens, counts, ws, n_ws = self._args(block_table, kv_lens, refs, stream)
        each = isinstance(add, torch.Tensor)
        more = _ints("add", add, 1, kv_lens.shape[0]) if each else None
        got = None if granted is None else _ints("granted", granted, 1, kv_lens.shape[0])
        _raise(_lib().kda_pages_extend_granted(d, more, 0 if each else int(add), table, lens,
                                               counts, got, ws, n_ws, _raw_stream(stream)),
               "kda_pages_extend")

    def free(self, slots, block_table, kv_lens, refs, stream=None):
        """Release the rows ``slots`` (int32, distinct)."""
        d, table, lens, counts, _, _ = self._args(block_table, kv_lens, refs, stream)
        _raise(_lib().kda_pages_free(d, _ints("slots", slots, 1), slots.shape[0], table, lens,
                                     counts, _raw_stream(stream)), "kda_pages_free")

    def compact(self, block_table, kv_lens, refs, stream=None):
        """Move the held pages to the lowest ids, in every pool, and rename them
        in the table.  Afterwards pages [0, held) are held and the rest free."""
        d, table, _, counts, ws, n_ws = self._args(block_table, kv_lens, refs, stream)
        _raise(_lib().kda_pages_compact(d, self._arr, len(self.pools), table, counts, ws, n_ws,
                                        _raw_stream(stream)), "kda_pages_compact")
