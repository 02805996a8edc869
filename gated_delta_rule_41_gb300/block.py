"""Thin ctypes binding of what stands around a mixing layer (C ABI in
include/kda.h): the gated linear recurrence, the norm of a layer's output with
its gate, the residual sum with the norm before the next layer, and activations
kept in 8 bits for the backward pass.

    o, ht, saved = gated_scan_fwd(x, g, save_for_backward=True)
    y, o8, z8 = gated_norm_fwd(o_heads, z_heads, w, keep8=True)
    res, n = add_norm_fwd(res, y @ w_out, w2, alpha=scale)
    ...
    grads = add_norm_bwd(res, w2, dn, dres, x=x_out, alpha=scale)
    grads = gated_norm_bwd(o8, z8, w, dy)
    grads = gated_scan_bwd(x, g, do, saved)

A step of a server calls the same norms, and ``gated_scan_step``.  As in
``kda.py`` every step runs in the library's kernels on the caller's stream;
nothing here waits for the GPU.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import kda as _kda
from .kda import KDA_BF16, KDA_F32, KdaError, _raise
from .paged import _fresh, _get_device, _raw_stream

GATES = {"sigmoid": 0, "silu": 1}
STATE_EVERY = 64      # tokens between the states that a saving scan keeps
SCALE_BLOCK = 32      # neighbours that share a scale


class KdaScanDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int),
                ("dtype", ctypes.c_int), ("tied", ctypes.c_int),
                ("x_batch", ctypes.c_longlong), ("x_token", ctypes.c_longlong),
                ("g_batch", ctypes.c_longlong), ("g_token", ctypes.c_longlong)]


class KdaGatedNormDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("w_dtype", ctypes.c_int), ("gate", ctypes.c_int),
                ("eps", ctypes.c_float), ("x_stride", ctypes.c_longlong),
                ("gate_stride", ctypes.c_longlong)]


class KdaAddNormDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("D", ctypes.c_int), ("dtype", ctypes.c_int),
                ("res_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("alpha", ctypes.c_float), ("r_stride", ctypes.c_longlong),
                ("x_stride", ctypes.c_longlong)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        lib = _kda.load_library()
        P, I, L, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
        C, G, A = (ctypes.POINTER(x) for x in (KdaScanDims, KdaGatedNormDims, KdaAddNormDims))
        for name, res, args in (
                ("kda_gated_scan_fwd", I, [C, P, I] + [P] * 7),
                ("kda_gated_scan_bwd", I, [C, P, I] + [P] * 10),
                ("kda_gated_scan_step", I, [C] + [P] * 6),
                ("kda_gated_norm_fwd", I, [G] + [P] * 9),
                ("kda_gated_norm_workspace_bytes", S, [G]),
                ("kda_gated_norm_bwd", I, [G] + [P] * 10 + [S, P]),
                ("kda_add_norm_fwd", I, [A] + [P] * 7),
                ("kda_add_norm_workspace_bytes", S, [A]),
                ("kda_add_norm_bwd", I, [A] + [P] * 11 + [S, P]),
                ("kda_pack8", I, [P, I, L, I, L, P, P, P]),
                ("kda_unpack8", I, [P, P, L, I, P, I, P]),
                ("kda_selftest_exchange", I, [I, I, I, I, L, L, P, P])):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _bound = lib
    return _bound


_CODES = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}


def _code(name, t):
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise KdaError(3, f"{name}: {t.dtype} (bf16 or fp32 only)") from None


def _sizes(shape):
    """The C entries take 32-bit sizes."""
    if any(n >= 1 << 31 for n in shape):
        raise KdaError(3, f"sizes {tuple(shape)} (below 2^31 each)")
    return shape


def _at(t):
    return None if t is None else t.data_ptr()


def _here(*tensors):
    """The kernels run on the current device, which is returned: so must their tensors be."""
    dev = torch.cuda.current_device() if _get_device is None else _get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise KdaError(1, "tensors must be CUDA tensors on the current device")
    return dev


def _given(grads, *names):
    """The tensors that a caller gives for a backward pass's results."""
    return () if grads is None else [grads.get(n) for n in names]


# What was found right and made for calls of these sizes, strides and types (and, where a workspace's
# size is a part of it, on this device: it goes by the SMs): a small call's time is the host's.
_plans = {}


def _plan(key, make):
    if len(_plans) >= 1024:
        _plans.clear()
    got = _plans[key] = make()
    return got


def _like(w):
    """What a plan knows of an optional tensor."""
    return None if w is None else (w.shape, w.stride(), w.dtype)


def _dense(name, t, shape, dtype=None):
    """The pointer of a contiguous CUDA tensor of this shape (and type)."""
    if t is None:
        return None
    if not t.is_cuda or t.shape != shape or not t.is_contiguous() \
            or (dtype is not None and t.dtype != dtype):
        raise KdaError(1, f"{name} must be a contiguous CUDA tensor {tuple(shape)}"
                          + (f" of {dtype}" if dtype is not None else ""))
    return t.data_ptr()


def _out(t, shape, dtype, like, stream, name="out"):
    if t is None:
        return _fresh(stream, shape, dtype, like.device)
    _dense(name, t, shape, dtype)
    return t


def _vector(name, w, D):
    """A parameter [D], float32 or bf16."""
    if w is None:
        return None
    if not w.is_cuda or w.shape != (D,) or not w.is_contiguous() or w.dtype not in _CODES:
        raise KdaError(1, f"{name} must be a contiguous CUDA tensor [{D}], float32 or bf16")
    return w.data_ptr()


# ---- 8 bits ----

class Packed8:
    """A tensor in 8 bits: ``codes`` float8_e4m3fn of its shape, and ``scales``
    uint8 [..., ceil(D / 32)], the exponents (+ 127) that blocks of 32
    neighbours along the last dimension share."""

    def __init__(self, codes, scales):
        if codes.dtype != torch.float8_e4m3fn or not codes.is_cuda or not codes.is_contiguous() \
                or codes.dim() < 1:
            raise KdaError(1, "codes must be a contiguous float8_e4m3fn CUDA tensor")
        want = codes.shape[:-1] + (-(-codes.shape[-1] // SCALE_BLOCK),)
        if scales.dtype != torch.uint8 or not scales.is_cuda or not scales.is_contiguous() \
                or scales.shape != want:
            raise KdaError(1, f"scales must be a contiguous uint8 CUDA tensor {tuple(want)}")
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return self.codes.shape

    @classmethod
    def empty(cls, shape, device, stream=None):
        shape = torch.Size(shape)
        return cls(_fresh(stream, shape, torch.float8_e4m3fn, device),
                   _fresh(stream, shape[:-1] + (-(-shape[-1] // SCALE_BLOCK),), torch.uint8, device))


def _rows(name, x):
    """x as rows of one stride: (rows, width, stride).  A strided tensor's
    contiguous last dimensions count as one where blocks do not cross them."""
    D = _sizes(x.shape[-1:])[0]
    n = x.numel() // D if D else 0
    if x.is_contiguous():
        return n, D, D
    if x.stride(-1) == 1 or D == 1:
        dims = [(s, st) for s, st in zip(x.shape[:-1], x.stride()[:-1]) if s > 1]
        width = D
        while D % SCALE_BLOCK == 0 and dims and dims[-1][1] == width \
                and width * dims[-1][0] < 1 << 31:
            width *= dims.pop()[0]
        run = dims[-1][1] if dims else width
        for s, st in reversed(dims):
            if st != run:
                break
            run = st * s
        else:
            return x.numel() // width, width, dims[-1][1] if dims else width
    raise KdaError(1, f"{name}: rows must be contiguous and equally far apart")


def pack8(x, out: Optional[Packed8] = None, stream=None) -> Packed8:
    """x [..., D] (bf16 or fp32; rows may lie apart) in 8 bits: blocks of 32
    neighbours share the smallest 2^e with max |x| <= 448 * 2^e, so a value is
    off by 2^-4 of itself at most (or 2^-10 of 2^e).  Infinities and NaN become
    NaN."""
    _here(x, *(() if out is None else (out.codes, out.scales)))
    lib, t = _lib(), _code("x", x)
    if not x.is_cuda or x.dim() < 1 or x.shape[-1] < 1:
        raise KdaError(1, "x must be a CUDA tensor [..., D]")
    rows, width, stride = _rows("x", x)
    if out is None:
        out = Packed8.empty(x.shape, x.device, stream)
    elif out.shape != x.shape:
        raise KdaError(1, "out has another shape than x")
    _raise(lib.kda_pack8(x.data_ptr(), t, rows, width, stride, out.codes.data_ptr(),
                         out.scales.data_ptr(), _raw_stream(stream)), "kda_pack8")
    return out


def unpack8(p: Packed8, dtype=torch.bfloat16, out=None, stream=None):
    """The values that ``p`` stands for, in fp32 (exact) or bf16 (exact down to its
    smallest steps, 2^-133: codes at the least scale reach 2^-135)."""
    _here(p.codes, p.scales, out)
    codes = p.codes
    D = codes.shape[-1]
    if D >= 1 << 31:
        _sizes(codes.shape[-1:])
    out = _out(out, codes.shape, dtype, codes, stream)
    st = _lib().kda_unpack8(codes.data_ptr(), p.scales.data_ptr(), codes.numel() // max(D, 1), D,
                            out.data_ptr(), _code("out", out), _raw_stream(stream))
    if st:
        _raise(st, "kda_unpack8")
    return out


# ---- the gated recurrence ----

def _scan(x, g, tied):
    key = ("scan", x.shape, x.stride(), x.dtype, g.shape, g.stride(), g.dtype, bool(tied))
    return _plans.get(key) or _plan(key, lambda: _scan_dims(x, g, tied))


def _scan_dims(x, g, tied):
    if x.dim() != 3 or g.shape != x.shape or g.dtype != x.dtype:
        raise KdaError(1, "x and g must be tensors [B, T, C] of one type")
    for n, t in (("x", x), ("g", g)):
        if t.stride(2) != 1 and t.shape[2] > 1:
            raise KdaError(1, f"{n} must have contiguous channels")
    B, T, C = _sizes(x.shape)
    return ctypes.pointer(KdaScanDims(B, T, C, _code("x", x), int(bool(tied)), x.stride(0), x.stride(1),
                                      g.stride(0), g.stride(1)))


def _scan_seqs(x, cu_seqlens):
    """Pointer of cu_seqlens, its sequences, and the rows of the states."""
    if cu_seqlens is None:
        return None, 0, x.shape[0]
    n = _kda._check_cu(cu_seqlens)
    return cu_seqlens.data_ptr(), n, n


def gated_scan_fwd(x, g, initial_state=None, output_final_state=False, tied=False, cu_seqlens=None,
                   save_for_backward=False, out=None, final_state=None, stream=None):
    """The gated linear recurrence h_t = exp(g_t) h_{t-1} + u_t x_t per channel,
    o_t = h_t, with u_t = 1, or 1 - exp(g_t) if ``tied``.  x, g [B, T, C] (bf16
    or fp32; slices of a wider projection will do), g a log-decay (<= 0).  Returns (o,
    final_state or None), plus the kept states when ``save_for_backward`` is
    set (pass them to ``gated_scan_bwd``).  ``initial_state`` and the final
    state are float32 [B, C]; with ``cu_seqlens`` (int32 [N + 1], B = 1) the
    sequences are packed along T and they are [N, C].  An infinite state may be a
    NaN from the next token on, in its channel and sequence."""
    _here(x, g, initial_state, cu_seqlens, out, final_state)
    lib, d = _lib(), _scan(x, g, tied)
    cu, n, rows = _scan_seqs(x, cu_seqlens)
    B, T, C = x.shape
    h0 = None if initial_state is None else _dense("initial_state", initial_state, (rows, C), torch.float32)
    out = _out(out, x.shape, x.dtype, x, stream)
    if output_final_state:
        final_state = _out(final_state, (rows, C), torch.float32, x, stream, "final_state")
    else:
        final_state = None
    saved = None
    if save_for_backward:
        saved = _fresh(stream, (B, -(-T // STATE_EVERY), C), torch.float32, x.device)
    st = lib.kda_gated_scan_fwd(d, cu, n, x.data_ptr(), g.data_ptr(), h0, out.data_ptr(),
                                _at(final_state), _at(saved), _raw_stream(stream))
    if st:
        _raise(st, "kda_gated_scan_fwd")
    return (out, final_state, saved) if save_for_backward else (out, final_state)


def gated_scan_bwd(x, g, do, saved=None, dht=None, initial_state=None, tied=False, cu_seqlens=None,
                   grads=None, stream=None):
    """Backward of ``gated_scan_fwd``.  Returns dict dx, dg, dh0 (dh0 with
    ``initial_state``).  ``saved`` are the states kept by the forward pass on
    the same inputs; without them they are computed again."""
    _here(x, g, do, saved, dht, initial_state, cu_seqlens, *_given(grads, "dx", "dg", "dh0"))
    lib, d = _lib(), _scan(x, g, tied)
    cu, n, rows = _scan_seqs(x, cu_seqlens)
    B, T, C = x.shape
    h0 = _dense("initial_state", initial_state, (rows, C), torch.float32)
    at = _dense("do", do, x.shape, x.dtype), _dense("dht", dht, (rows, C), torch.float32)
    if grads is None:
        grads = dict(dx=_fresh(stream, x.shape, x.dtype, x.device),
                     dg=_fresh(stream, x.shape, x.dtype, x.device),
                     dh0=None if initial_state is None
                     else _fresh(stream, (rows, C), torch.float32, x.device))
    to = (_dense("dx", grads["dx"], x.shape, x.dtype), _dense("dg", grads["dg"], x.shape, x.dtype),
          _dense("dh0", grads.get("dh0"), (rows, C), torch.float32))
    states, s = (B, -(-T // STATE_EVERY), C), _raw_stream(stream)
    if saved is None:
        saved = _fresh(stream, states, torch.float32, x.device)
        _raise(lib.kda_gated_scan_fwd(d, cu, n, x.data_ptr(), g.data_ptr(), h0, None, None,
                                      saved.data_ptr(), s), "kda_gated_scan_fwd")
    _raise(lib.kda_gated_scan_bwd(d, cu, n, x.data_ptr(), g.data_ptr(), h0,
                                  _dense("saved", saved, states, torch.float32), *at, *to, s),
           "kda_gated_scan_bwd")
    return grads


def gated_scan_step(x, g, state, tied=False, new_state=None, out=None, stream=None):
    """One token of the recurrence: x, g [B, C], ``state`` [B, C] float32, updated
    in place (or left, where ``new_state`` takes the new one).  Returns o
    [B, C]."""
    _here(x, g, state, new_state, out)
    key = ("step", x.shape, x.stride(), x.dtype, g.shape, g.stride(), g.dtype, bool(tied))
    d = _plans.get(key) or _plan(key, lambda: _step_dims(x, g, tied))
    h = _dense("state", state, x.shape, torch.float32)
    to = h if new_state is None else _dense("new_state", new_state, x.shape, torch.float32)
    out = _out(out, x.shape, x.dtype, x, stream)
    st = _lib().kda_gated_scan_step(d, x.data_ptr(), g.data_ptr(), h, to, out.data_ptr(),
                                    _raw_stream(stream))
    if st:
        _raise(st, "kda_gated_scan_step")
    return out


def _step_dims(x, g, tied):
    if x.dim() != 2 or g.shape != x.shape or g.dtype != x.dtype:
        raise KdaError(1, "x and g must be tensors [B, C] of one type")
    for n, t in (("x", x), ("g", g)):
        if t.stride(1) != 1 and t.shape[1] > 1:
            raise KdaError(1, f"{n} must have contiguous channels")
    B, C = _sizes(x.shape)
    return ctypes.pointer(KdaScanDims(B, 1, C, _code("x", x), int(bool(tied)), x.stride(0), C,
                                      g.stride(0), C))


# ---- the norms ----

def _heads(name, t, shape):
    """Token stride of a tensor [T, H, D] whose tokens may lie apart."""
    T, H, D = shape
    if not t.is_cuda or t.shape != shape:
        raise KdaError(1, f"{name} must be a CUDA tensor {tuple(shape)}")
    a, b, c = t.stride()
    if (c != 1 and D > 1) or (H > 1 and b != D):
        raise KdaError(1, f"{name}: the heads of a token must be contiguous")
    return a if T > 1 else H * D


def _gated_dims(x, gate, weight, dtype, eps, act):
    if act not in GATES:
        raise KdaError(1, f"gate {act!r} (sigmoid or silu)")
    T, H, D = _sizes(x.shape)
    packed = isinstance(x, Packed8)
    return KdaGatedNormDims(
        T, H, D, dtype, KDA_BF16 if weight is not None and weight.dtype == torch.bfloat16 else KDA_F32,
        GATES[act], eps, H * D if packed else _heads("x", x, x.shape),
        H * D if packed else _heads("gate", gate, x.shape))


def gated_norm_fwd(x, gate, weight=None, eps=1e-5, act="sigmoid", keep8=False, out=None, stream=None):
    """The norm of a layer's output with its gate: y = weight s(gate) x /
    sqrt(mean(x^2) + eps) over the last dimension of x [T, H, D] (bf16 or fp32;
    tokens may lie apart, as those of gate), s = sigmoid or z sigmoid(z)
    (``act`` "silu").  ``weight`` [D] is shared by the heads.  Returns y, or with
    ``keep8`` (y, x, gate) with the inputs as ``Packed8`` for
    ``gated_norm_bwd``."""
    _here(x, gate, weight, out)
    key = ("gated", x.shape, x.stride(), x.dtype, gate.shape, gate.stride(), gate.dtype, _like(weight),
           eps, act)
    d = _plans.get(key) or _plan(key, lambda: _gated_fwd_dims(x, gate, weight, eps, act))
    y = _out(out, x.shape, x.dtype, x, stream)
    kept = [Packed8.empty(x.shape, x.device, stream) for _ in range(2)] if keep8 else []
    ptrs = [t.data_ptr() for p in kept for t in (p.codes, p.scales)] or (None,) * 4
    st = _lib().kda_gated_norm_fwd(d, x.data_ptr(), gate.data_ptr(), _at(weight), y.data_ptr(), *ptrs,
                                   _raw_stream(stream))
    if st:
        _raise(st, "kda_gated_norm_fwd")
    return (y, *kept) if keep8 else y


def _gated_fwd_dims(x, gate, weight, eps, act):
    if x.dim() != 3 or gate.dtype != x.dtype:
        raise KdaError(1, "x and gate must be tensors [T, H, D] of one type")
    _vector("weight", weight, x.shape[2])
    return ctypes.pointer(_gated_dims(x, gate, weight, _code("x", x), eps, act))


def _workspace(need, workspace, like, stream):
    if need and workspace is not None and not workspace.is_contiguous():
        raise KdaError(1, "workspace must be a contiguous CUDA tensor")
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        return workspace
    return _fresh(stream, max(need, 1), torch.uint8, like.device)


def gated_norm_bwd(x, gate, weight, dy, eps=1e-5, act="sigmoid", workspace=None, grads=None, stream=None):
    """Backward of ``gated_norm_fwd``: dict dx, dgate (dy's type), dw (float32).
    (``workspace``, for dw: calls that may overlap need one each; without, a call makes its own.)
    x and gate as given to the forward pass, or both as the ``Packed8`` that it
    kept; then the gradients are those at the values that these stand for."""
    packed = isinstance(x, Packed8)
    if packed != isinstance(gate, Packed8):
        raise KdaError(1, "x and gate must both be Packed8, or neither")
    src = (x.codes, x.scales, gate.codes, gate.scales) if packed else (x, None, gate, None)
    dev = _here(*src, weight, dy, workspace, *_given(grads, "dx", "dgate", "dw"))
    lib = _lib()
    key = ("gated_bwd", dev, packed, src[0].shape, src[0].stride(), src[0].dtype, src[2].shape, src[2].stride(),
           src[2].dtype, _like(weight), dy.dtype, eps, act)
    d, need = _plans.get(key) or _plan(key, lambda: _gated_bwd_dims(x, gate, weight, dy, eps, act, packed))
    D = x.shape[2]
    w, up = _at(weight), _dense("dy", dy, x.shape)
    if grads is None:
        grads = dict(dx=_fresh(stream, x.shape, dy.dtype, dy.device),
                     dgate=_fresh(stream, x.shape, dy.dtype, dy.device),
                     dw=None if weight is None else _fresh(stream, (D,), torch.float32, dy.device))
    to = (_dense("dx", grads["dx"], x.shape, dy.dtype), _dense("dgate", grads["dgate"], x.shape, dy.dtype),
          _dense("dw", grads.get("dw"), (D,), torch.float32))
    need = need if to[2] is not None else 0
    ws = _workspace(need, workspace, dy, stream)
    _raise(lib.kda_gated_norm_bwd(d, *(_at(t) for t in src), w, up, *to, ws.data_ptr(), need,
                                  _raw_stream(stream)), "kda_gated_norm_bwd")
    return grads


def _gated_bwd_dims(x, gate, weight, dy, eps, act, packed):
    if len(x.shape) != 3 or gate.shape != x.shape:
        raise KdaError(1, "x and gate must be [T, H, D]")
    if not packed and (x.dtype != dy.dtype or gate.dtype != dy.dtype):
        raise KdaError(1, "x, gate and dy must have one type")
    _vector("weight", weight, x.shape[2])
    d = ctypes.pointer(_gated_dims(x, gate, weight, _code("dy", dy), eps, act))
    return d, int(_lib().kda_gated_norm_workspace_bytes(d))


def _tokens2(name, t, T, D):
    """Token stride of a tensor [T, D] whose tokens may lie apart."""
    if not t.is_cuda or t.shape != (T, D) or (t.stride(1) != 1 and D > 1):
        raise KdaError(1, f"{name} must be a CUDA tensor [{T}, {D}] with contiguous rows")
    return t.stride(0) if T > 1 else D


def _add_dims(residual, x, weight, alpha, dtype, eps):
    if residual.dim() != 2:
        raise KdaError(1, "residual must be a tensor [T, D]")
    T, D = _sizes(residual.shape)
    vec = isinstance(alpha, torch.Tensor)
    w = _vector("weight", weight, D)
    av = _vector("alpha", alpha, D) if vec else None
    if weight is not None and vec and weight.dtype != alpha.dtype:
        raise KdaError(1, "weight and alpha must have one type")
    p = weight if weight is not None else alpha if vec else None
    return KdaAddNormDims(
        T, D, dtype, _code("residual", residual),
        KDA_BF16 if p is not None and p.dtype == torch.bfloat16 else KDA_F32, eps,
        1.0 if vec or alpha is None else float(alpha), _tokens2("residual", residual, T, D),
        D if x is None else _tokens2("x", x, T, D)), w, av


def add_norm_fwd(residual, x, weight=None, alpha=None, eps=1e-5, out=None, out_residual=None, stream=None):
    """The residual sum and the norm before the next layer: r = residual + alpha x,
    y = weight r / sqrt(mean(r^2) + eps) over the last dimension of [T, D].
    ``alpha`` is a number or a vector [D] (None: 1); x may be None (the norm
    alone).  The residual stream may be fp32 beside bf16 x.  Returns (r, y);
    ``out_residual`` may be ``residual`` itself.  (y is of x's type, without x
    of ``out``'s or the residual's.)"""
    _here(residual, x, weight, alpha if isinstance(alpha, torch.Tensor) else None, out, out_residual)
    like = x if x is not None else out if out is not None else residual
    vec = isinstance(alpha, torch.Tensor)
    key = ("add", residual.shape, residual.stride(), residual.dtype, _like(x), _like(weight),
           _like(alpha) if vec else alpha, like.dtype, eps)
    d = _plans.get(key) or _plan(key, lambda: ctypes.pointer(
        _add_dims(residual, x, weight, alpha, _code("x", like), eps)[0]))
    y = _out(out, residual.shape, like.dtype, residual, stream)
    r = out_residual
    if x is not None or r is not None:
        r = _out(r, residual.shape, residual.dtype, residual, stream, "out_residual")
    st = _lib().kda_add_norm_fwd(d, residual.data_ptr(), _at(x), alpha.data_ptr() if vec else None,
                                 _at(weight), _at(r), y.data_ptr(), _raw_stream(stream))
    if st:
        _raise(st, "kda_add_norm_fwd")
    return (residual if r is None else r), y


def _add_bwd_dims(residual, weight, dy, x, alpha, eps):
    d, _, av = _add_dims(residual, x, weight, alpha, _code("dy", dy), eps)
    if av is not None and x is None:
        raise KdaError(1, "a vector alpha needs x")
    if x is not None and x.dtype != dy.dtype:
        raise KdaError(1, "x and dy must have one type")
    d = ctypes.pointer(d)
    return d, int(_lib().kda_add_norm_workspace_bytes(d))


def add_norm_bwd(residual, weight, dy, dres=None, x=None, alpha=None, eps=1e-5, workspace=None,
                 grads=None, stream=None):
    """Backward of ``add_norm_fwd``.  ``residual`` is the r that it returned,
    ``dy`` the gradient of y, ``dres`` that of r from what else reads it.
    Returns dict dres (of the residual that went in), dx = alpha dres, dw and
    dalpha (float32; dalpha for a vector alpha, which needs the forward's x).
    Without alpha, and in one type, dx is the tensor dres itself, as it may be in ``grads``.  (``workspace`` as for
    ``gated_norm_bwd``.)"""
    dev = _here(residual, weight, dy, dres, x, alpha if isinstance(alpha, torch.Tensor) else None, workspace,
                *_given(grads, "dres", "dx", "dw", "dalpha"))
    lib = _lib()
    vec = isinstance(alpha, torch.Tensor)
    key = ("add_bwd", dev, residual.shape, residual.stride(), residual.dtype, _like(x), _like(weight),
           _like(alpha) if vec else alpha, dy.dtype, eps)
    d, need = _plans.get(key) or _plan(key, lambda: _add_bwd_dims(residual, weight, dy, x, alpha, eps))
    D = residual.shape[1]
    w, av = _at(weight), alpha.data_ptr() if vec else None
    at = _dense("dy", dy, residual.shape), _dense("dres", dres, residual.shape, residual.dtype)
    if grads is None:
        one = alpha is None and dy.dtype == residual.dtype
        grads = dict(dres=_fresh(stream, residual.shape, residual.dtype, dy.device),
                     dx=None if one else _fresh(stream, residual.shape, dy.dtype, dy.device),
                     dw=None if weight is None else _fresh(stream, (D,), torch.float32, dy.device),
                     dalpha=None if av is None else _fresh(stream, (D,), torch.float32, dy.device))
    else:
        one = residual.numel() > 0 and _at(grads.get("dx")) == _at(grads["dres"])
        if one and alpha is not None and (vec or alpha != 1):
            raise KdaError(1, "dx and dres are one tensor")
    to = (_dense("dres", grads["dres"], residual.shape, residual.dtype),
          _dense("dx", grads.get("dx"), residual.shape, dy.dtype) if not one else None,
          _dense("dw", grads.get("dw"), (D,), torch.float32),
          _dense("dalpha", grads.get("dalpha"), (D,), torch.float32))
    if to[3] is not None and x is None:
        raise KdaError(1, "dalpha needs x")
    need = need if to[2] is not None or to[3] is not None else 0
    ws = _workspace(need, workspace, dy, stream)
    _raise(lib.kda_add_norm_bwd(d, residual.data_ptr(), _at(x), av, w, *at, *to, ws.data_ptr(), need,
                                _raw_stream(stream)), "kda_add_norm_bwd")
    if one:
        grads["dx"] = grads["dres"]
    return grads
