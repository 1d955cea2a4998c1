"""Binding of the sequence-layer operators (layer norm, linear, delta rule) of include/zsolve.h.

As in the rest of the binding, a function with a C entry point's name calls it
on tensors that the caller holds; `Seq` owns a handle, allocates the outputs
and runs on torch's current stream.
"""
from __future__ import annotations

import ctypes

from . import ZSOLVE_ETIMEOUT, ZSOLVE_OK, ZsolveError, _lib

ZSOLVE_F32 = 0
ZSOLVE_BF16 = 1
ZSOLVE_F16 = 2

ZSOLVE_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


torch = None  # imported with the first handle: the rest of the package loads without it
_TYPES = {}
_device = None  # torch's current device, an index
_only = -2  # the device of a process that has one, where no tensor is on another


def _use_torch():
    global torch, _device, _only
    if torch is None:
        import torch as module
        torch = module
        _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        if torch.cuda.device_count() == 1:
            _only = 0
        _TYPES.update({torch.float32: ZSOLVE_F32, torch.bfloat16: ZSOLVE_BF16, torch.float16: ZSOLVE_F16})


def _type(t, name) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32, bfloat16 or float16, got {t.dtype}")
    return code


def _cuda(t, name):
    """Refuses a tensor that is not on the current device, which the library holds to be the handle's."""
    if t.get_device() != _device():
        raise ValueError(f"{name}: expected a CUDA tensor on the current device, {_device()}, got one on {t.device}")


def _rows(t, name, dtype=None, shape=None):
    """(pointer, rows, d, row stride) of a matrix: a tensor (..., d) whose rows lie at one distance."""
    if t.get_device() != _only:
        _cuda(t, name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    size = t.shape
    if len(size) != 2:
        if not size:
            raise ValueError(f"{name}: expected rows of values")
        t = _flat(t, name)
        size = t.shape
    m, d = size
    if shape is not None and shape != (m, d):
        raise ValueError(f"{name}: expected {shape[0]} rows of {shape[1]}, got {m} of {d}")
    ld, one = t.stride()
    if one != 1 and d > 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    return t.data_ptr(), m, d, ld if m > 1 else max(d, 1)


def _flat(t, name):
    if not t.numel():
        return t.reshape(-1, t.shape[-1])
    try:
        return t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: the rows must lie at one distance") from None


def _vector(t, name, n, dtype, shape=None, last=0):
    """Pointer of n contiguous values, or 0 for None; with a shape, in its order, of which `last` sizes are a token's."""
    if t is None:
        return 0
    if t.get_device() != _only:
        _cuda(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is None or t.shape != shape:
        if t.numel() != n:
            raise ValueError(f"{name}: expected {n} contiguous values, got {tuple(t.shape)}")
        if shape is not None:
            _same_order(t, name, shape, last)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous values, got {tuple(t.shape)}")
    return t.data_ptr()


def _same_order(t, name, shape, last):
    """Refuses a shape of as many values whose order is not that of `shape`: it is flat, or ends as `shape` does and,
    with as many sizes before the last ones, begins so too."""
    dim = t.dim()
    if dim < 2:
        return
    j = min(last, dim - 1)
    if (j and t.shape[-j:] != shape[-j:]) or (dim == len(shape) and t.shape != shape):
        raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(t.shape)}")


def _current_stream() -> int:
    """The handle of torch's current stream on the current device."""
    try:  # without making a Stream object, where torch offers that
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _check_seq(seq, status):
    if status != ZSOLVE_OK:
        msg = _lib.zsolve_seq_last_error(seq).decode() if seq else ""
        raise ZsolveError(status, f"{_lib.zsolve_strerror(status).decode()}: {msg}")


# ---------------------------------------------------------------- C entry points


def zsolve_seq_create() -> ctypes.c_void_p:
    _use_torch()
    seq = ctypes.c_void_p()
    _check_seq(None, _lib.zsolve_seq_create(ctypes.byref(seq)))
    return seq


def zsolve_seq_set_stream(seq, stream=None) -> None:
    """stream: a torch.cuda.Stream, a raw handle, or None for torch's current stream."""
    if stream is None:
        stream = torch.cuda.current_stream()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check_seq(seq, _lib.zsolve_seq_set_stream(seq, handle))


def zsolve_seq_reserve(seq, nbytes: int) -> None:
    _check_seq(seq, _lib.zsolve_seq_reserve(seq, int(nbytes)))


def zsolve_seq_workspace_bytes(seq) -> int:
    return int(_lib.zsolve_seq_workspace_bytes(seq))


def zsolve_seq_launches(seq) -> int:
    return int(_lib.zsolve_seq_launches(seq))


def zsolve_seq_last_error(seq) -> str:
    return _lib.zsolve_seq_last_error(seq).decode()


def zsolve_seq_check(seq) -> None:
    _check_seq(seq, _lib.zsolve_seq_check(seq))


def zsolve_seq_destroy(seq) -> None:
    _lib.zsolve_seq_destroy(seq)


def _norm_weights(x, w, b):
    """Type code of w and b (the type of x, or float32), and their torch type."""
    given = w if w is not None else b
    dt = x.dtype if given is None else given.dtype
    if dt not in (x.dtype, torch.float32):
        raise TypeError(f"w and b: expected {x.dtype} or torch.float32, got {dt}")
    return dt


def zsolve_layernorm(seq, x, w, b, eps, y, mean=None, rstd=None) -> None:
    """y <- layer norm of the rows of x (..., d); w, b: (d,) or None; mean, rstd: float32, one value a row, or None."""
    xp, m, d, ldx = _rows(x, "x")
    yp, _, _, ldy = _rows(y, "y", x.dtype, (m, d))
    wt = _norm_weights(x, w, b)
    rows = (m,) if x.dim() == 2 else x.shape[:-1]
    _check_seq(seq, _lib.zsolve_layernorm(seq, _type(x, "x"), _TYPES[wt], m, d, xp, ldx, _vector(w, "w", d, wt),
                                          _vector(b, "b", d, wt), eps, yp, ldy,
                                          _vector(mean, "mean", m, torch.float32, rows),
                                          _vector(rstd, "rstd", m, torch.float32, rows)))


def zsolve_layernorm_bwd(seq, dy, x, mean, rstd, w, dx, dw=None, db=None) -> None:
    """dx (the shape of x), dw and db (the type of w, or of x without one; None: not formed) from dy."""
    xp, m, d, ldx = _rows(x, "x")
    dyp, _, _, lddy = _rows(dy, "dy", x.dtype, (m, d))
    dxp, _, _, lddx = _rows(dx, "dx", x.dtype, (m, d))
    wt = _norm_weights(x, w, dw if dw is not None else db)
    rows = (m,) if x.dim() == 2 else x.shape[:-1]
    _check_seq(seq, _lib.zsolve_layernorm_bwd(seq, _type(x, "x"), _TYPES[wt], m, d, dyp, lddy, xp, ldx,
                                              _vector(mean, "mean", m, torch.float32, rows),
                                              _vector(rstd, "rstd", m, torch.float32, rows), _vector(w, "w", d, wt), dxp,
                                              lddx, _vector(dw, "dw", d, wt), _vector(db, "db", d, wt)))


def _act(act) -> int:
    if act not in ZSOLVE_ACTS:
        raise ValueError(f"act: expected one of {', '.join(ZSOLVE_ACTS)}, got {act!r}")
    return ZSOLVE_ACTS[act]


def _optional_rows(t, name, dtype, shape):
    """(pointer, row stride) of a matrix, or zeros for None."""
    if t is None:
        return 0, 0
    p, _, _, ld = _rows(t, name, dtype, shape)
    return p, ld


def zsolve_linear(seq, x, w, b, act, r, y, z=None) -> None:
    """y <- act(x w^T + b) + r; x (..., k), w (n, k), b (n,) or None, r and y (..., n), r or None; z: as y, or None."""
    xp, m, k, ldx = _rows(x, "x")
    wp, n, _, ldw = _rows(w, "w", x.dtype, (w.shape[0], k))
    rp, ldr = _optional_rows(r, "r", x.dtype, (m, n))
    yp, _, _, ldy = _rows(y, "y", x.dtype, (m, n))
    zp, ldz = _optional_rows(z, "z", x.dtype, (m, n))
    _check_seq(seq, _lib.zsolve_linear(seq, _type(x, "x"), m, n, k, xp, ldx, wp, ldw, _vector(b, "b", n, x.dtype),
                                       _act(act), rp, ldr, yp, ldy, zp, ldz))


def zsolve_linear_bwd(seq, dy, x, w, act, z, dx=None, dw=None, db=None) -> None:
    """dx, dw and db (shapes of x, w and the bias; None: not formed) from dy; z: as zsolve_linear kept it."""
    xp, m, k, ldx = _rows(x, "x")
    wp, n, _, ldw = _rows(w, "w", x.dtype, (w.shape[0], k))
    dyp, _, _, lddy = _rows(dy, "dy", x.dtype, (m, n))
    zp, ldz = _optional_rows(z, "z", x.dtype, (m, n))
    dxp, lddx = _optional_rows(dx, "dx", x.dtype, (m, k))
    dwp, lddw = _optional_rows(dw, "dw", x.dtype, (n, k))
    _check_seq(seq, _lib.zsolve_linear_bwd(seq, _type(x, "x"), m, n, k, dyp, lddy, xp, ldx, wp, ldw, _act(act), zp,
                                           ldz, dxp, lddx, dwp, lddw, _vector(db, "db", n, x.dtype)))


class zsolve_delta_args(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("hk", ctypes.c_int), ("hv", ctypes.c_int), ("dk", ctypes.c_int),
                ("dv", ctypes.c_int), ("nseq", ctypes.c_int), ("tokens", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("ldk", ctypes.c_int64), ("ldv", ctypes.c_int64),
                ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("s0", ctypes.c_void_p),
                ("scale", ctypes.c_double)]


def _tokens(t, name, dtype=None, shape=None, like=None):
    """(pointer, tokens, heads, d, token stride) of a tensor (tokens, heads, d) or (sequences, tokens, heads, d); with
    `like`, of its sequences x tokens."""
    if t.get_device() != _only:
        _cuda(t, name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() == 4:
        if like is not None and like.dim() == 4 and t.shape[:2] != like.shape[:2]:
            raise ValueError(f"{name}: expected the tokens {tuple(like.shape[:2])}, got {tuple(t.shape[:2])}")
        try:
            t = t.flatten(0, 1) if t.numel() == 0 else t.view((-1,) + t.shape[2:])
        except RuntimeError:
            raise ValueError(f"{name}: the tokens must lie at one distance") from None
    if t.dim() != 3:
        raise ValueError(f"{name}: expected tokens x heads x values, got {tuple(t.shape)}")
    n, h, d = t.shape
    if shape is not None and (n, h, d) != shape:
        raise ValueError(f"{name}: expected {shape[0]} x {shape[1]} x {shape[2]}, got {n} x {h} x {d}")
    if t.numel() and ((d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}: the heads of a token must be packed")
    return t.data_ptr(), n, h, d, t.stride(0) if n > 1 else h * d


def _delta_args(q, k, v, g, beta, s0, offsets, scale, nseq=None):
    qp, n, hk, dk, ldq = _tokens(q, "q")
    kp, _, _, _, ldk = _tokens(k, "k", q.dtype, (n, hk, dk), q)
    vp, _, hv, dv, ldv = _tokens(v, "v", q.dtype)
    lead = q.shape[:-2]
    if v.shape[:-2] != lead:
        raise ValueError(f"v: expected the tokens of q, {tuple(lead)}, got {tuple(v.shape[:-2])}")
    if offsets is not None:
        nseq = offsets.numel() - 1
        if nseq < 0:
            raise ValueError("offsets: expected one more than the sequences")
    elif nseq is None:
        nseq = q.shape[0] if q.dim() == 4 else 1
    gates = (*lead, hv)
    a = zsolve_delta_args(_type(q, "q"), hk, hv, dk, dv, nseq, n,
                          _vector(offsets, "offsets", nseq + 1, torch.int64) or None, qp, kp, vp, ldq, ldk, ldv,
                          _vector(g, "g", n * hv, torch.float32, gates, 1),
                          _vector(beta, "beta", n * hv, torch.float32, gates, 1),
                          _vector(s0, "s0", nseq * hv * dk * dv, torch.float32, (nseq, hv, dk, dv), 3),
                          dk ** -0.5 if scale is None else scale)
    return a


def zsolve_delta(seq, q, k, v, g, beta, o, s=None, s0=None, offsets=None, scale=None) -> None:
    """o, s <- the gated delta rule over whole sequences.

    q, k: (tokens, hk, dk), v, o: (tokens, hv, dv), g, beta: float32 (tokens, hv); or with two leading
    dimensions, sequences x tokens.  offsets: int64 (sequences + 1,) for sequences of different lengths in the
    packed form (without: one sequence).  s0, s: float32 (sequences, hv, dk, dv) or None; s may be s0.
    scale: 1 / sqrt(dk) unless given.
    """
    a = _delta_args(q, k, v, g, beta, s0, offsets, scale)
    op, _, _, _, ldo = _tokens(o, "o", q.dtype, (a.tokens, a.hv, a.dv), v)
    _check_seq(seq, _lib.zsolve_delta(seq, ctypes.byref(a), op, ldo, _state(s, a)))


def zsolve_delta_step(seq, q, k, v, g, beta, o, s=None, s0=None, offsets=None, scale=None) -> None:
    """As zsolve_delta, token by token: for one or a few tokens a sequence."""
    _step(seq, q, k, v, g, beta, o, s, s0, offsets, scale)


def _step(seq, q, k, v, g, beta, o, s, s0, offsets, scale, nseq=None):
    a = _delta_args(q, k, v, g, beta, s0, offsets, scale, nseq)
    op, _, _, _, ldo = _tokens(o, "o", q.dtype, (a.tokens, a.hv, a.dv), v)
    _check_seq(seq, _lib.zsolve_delta_step(seq, ctypes.byref(a), op, ldo, _state(s, a)))


def zsolve_delta_bwd(seq, dout, q, k, v, g, beta, dq, dk, dv, dg, dbeta, ds0=None, s0=None, ds=None, offsets=None,
                     scale=None) -> None:
    """dq .. dbeta and ds0 (shapes of q .. beta and s0, contiguous) from dout (as o) and ds (as s, or None)."""
    a = _delta_args(q, k, v, g, beta, s0, offsets, scale)
    op, _, _, _, lddo = _tokens(dout, "dout", q.dtype, (a.tokens, a.hv, a.dv), v)
    nk, nv, n = a.tokens * a.hk * a.dk, a.tokens * a.hv * a.dv, a.tokens * a.hv
    _check_seq(seq, _lib.zsolve_delta_bwd(seq, ctypes.byref(a), op, lddo, _state(ds, a), 
                                          _vector(dq, "dq", nk, q.dtype, q.shape, 2),
                                          _vector(dk, "dk", nk, q.dtype, k.shape, 2),
                                          _vector(dv, "dv", nv, q.dtype, v.shape, 2),
                                          _vector(dg, "dg", n, torch.float32, g.shape, 1),
                                          _vector(dbeta, "dbeta", n, torch.float32, beta.shape, 1), _state(ds0, a)))


def _state(s, a):
    return _vector(s, "s", a.nseq * a.hv * a.dk * a.dv, torch.float32, (a.nseq, a.hv, a.dk, a.dv), 3)


def _records(*tensors) -> bool:
    """Whether autograd is to record a call on these tensors."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _autograd():
    from . import seq_autograd
    return seq_autograd


class Seq:
    """Owns one handle of the sequence-layer operators; runs on torch's current stream.

    The calls enqueue their work and return.  A device-side wait that gives up (after about a second, so
    never on a GPU that works) leaves outputs that are not to be used: check() and close() raise for it.

    Example (x: bfloat16 CUDA tensor, tokens x d)::

        with Seq() as s:
            h, mean, rstd = s.layernorm(x, w, b)
            dx, dw, db = s.layernorm_bwd(dh, x, mean, rstd, w)

    Tensors that require gradients may be given as well: y of layernorm and linear and both outputs of delta then
    carry them (the handle has to be open in the backward pass).  mean, rstd and z carry none, nor does delta_step:
    a backward pass that needs theirs raises.
    """

    def __init__(self):
        self.seq = zsolve_seq_create()

    def _on_stream(self):
        _check_seq(self.seq, _lib.zsolve_seq_set_stream(self.seq, _current_stream()))

    def layernorm(self, x, w=None, b=None, eps=1e-5):
        """Returns (y, mean, rstd); mean and rstd are float32, for layernorm_bwd."""
        if _records(x, w, b):
            return _autograd().LayerNorm.apply(self, x, w, b, eps)
        self._on_stream()
        y = torch.empty_like(x)
        rows = x.shape[:-1]
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
        zsolve_layernorm(self.seq, x, w, b, eps, y, mean, rstd)
        return y, mean, rstd

    def layernorm_bwd(self, dy, x, mean, rstd, w=None):
        """Returns (dx, dw, db); dw and db have the type of w (of x without one)."""
        self._on_stream()
        dx = torch.empty_like(x)
        dt = x.dtype if w is None else w.dtype
        dw = torch.empty(x.shape[-1], dtype=dt, device=x.device)
        db = torch.empty(x.shape[-1], dtype=dt, device=x.device)
        zsolve_layernorm_bwd(self.seq, dy, x, mean, rstd, w, dx, dw, db)
        return dx, dw, db

    def linear(self, x, w, b=None, act="none", r=None, keep=False):
        """y = act(x w^T + b) + r; with keep=True (y, z), z for linear_bwd."""
        if _records(x, w, b, r):
            return _autograd().Linear.apply(self, x, w, b, act, r, keep)
        self._on_stream()
        shape = x.shape[:-1] + w.shape[:1]
        y = torch.empty(shape, dtype=x.dtype, device=x.device)
        z = torch.empty(shape, dtype=x.dtype, device=x.device) if keep else None
        zsolve_linear(self.seq, x, w, b, act, r, y, z)
        return (y, z) if keep else y

    def linear_bwd(self, dy, x, w, z=None, act="none"):
        """Returns (dx, dw, db); z as linear(keep=True) returned it (not needed without an activation)."""
        self._on_stream()
        dx = torch.empty_like(x)
        dw = torch.empty_like(w)
        db = torch.empty(w.shape[:1], dtype=x.dtype, device=x.device)
        zsolve_linear_bwd(self.seq, dy, x, w, act, z, dx, dw, db)
        return dx, dw, db

    def delta(self, q, k, v, g, beta, s0=None, offsets=None, scale=None):
        """Returns (o, s): the gated delta rule over whole sequences, from the states s0 (zero without) to s.

        Shapes as for zsolve_delta; s is (sequences, hv, dk, dv) float32.
        """
        if _records(q, k, v, g, beta, s0):
            return _autograd().Delta.apply(self, q, k, v, g, beta, s0, offsets, scale)
        self._on_stream()
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        nseq = offsets.numel() - 1 if offsets is not None else q.shape[0] if q.dim() == 4 else 1
        s = torch.empty((nseq, v.shape[-2], q.shape[-1], v.shape[-1]), dtype=torch.float32, device=v.device)
        zsolve_delta(self.seq, q, k, v, g, beta, o, s, s0, offsets, scale)
        return o, s

    def delta_bwd(self, dout, q, k, v, g, beta, s0=None, ds=None, offsets=None, scale=None):
        """Returns (dq, dk, dv, dg, dbeta, ds0) from the gradients of o and, unless None, of s."""
        self._on_stream()
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
        nseq = offsets.numel() - 1 if offsets is not None else q.shape[0] if q.dim() == 4 else 1
        ds0 = torch.empty((nseq, v.shape[-2], q.shape[-1], v.shape[-1]), dtype=torch.float32, device=v.device)
        zsolve_delta_bwd(self.seq, dout, q, k, v, g, beta, dq, dk, dv, dg, dbeta, ds0, s0, ds, offsets, scale)
        return dq, dk, dv, dg, dbeta, ds0

    def delta_step(self, q, k, v, g, beta, s, s_out=None, scale=None):
        """Returns (o, s): the next token of every sequence, q (sequences, hk, dk) and so on (or the next few,
        with two leading dimensions).  The states are updated in place, or written to s_out."""
        if _records(q, k, v, g, beta, s):
            return _autograd().Step.apply(self, q, k, v, g, beta, s, s if s_out is None else s_out, scale)
        self._on_stream()
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        s_out = s if s_out is None else s_out
        _step(self.seq, q, k, v, g, beta, o, s_out, s, None, scale, q.shape[0])
        return o, s_out

    def check(self):
        """Waits for the handle's work; raises if a device-side wait has given up since the last check."""
        zsolve_seq_check(self.seq)

    def close(self):
        """Releases the handle (after the work in flight); raises, once released, as check() does."""
        if not self.seq:
            return
        error = None
        try:
            zsolve_seq_check(self.seq)
        except ZsolveError as e:
            error = e if e.status == ZSOLVE_ETIMEOUT else None  # what else fails here is not the outputs'
        zsolve_seq_destroy(self.seq)
        self.seq = None
        if error is not None:
            raise error

    def __enter__(self):
        return self

    def __exit__(self, kind, *exc):
        try:
            self.close()
        except ZsolveError:
            if kind is None:  # else the block's own exception goes on
                raise

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
