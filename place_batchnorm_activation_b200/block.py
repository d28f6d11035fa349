"""Python binding of include/iabn_block.h: the row operators for transformer
blocks (block norm, gated activation, 8-bit checkpoints).

Argument marshalling only, as in the package's ``__init__``, which exports
everything here.  Tensors are [..., cols], a token a row; outputs are buffers
of the caller.  8-bit codes are ``torch.float8_e4m3fn`` or ``torch.int8``
tensors (the type names the format) of the shape of what they keep, scales
float32 [rows, ceil(cols / 128)].

Every call checks the shapes, types and devices of its tensors and raises
``IabnError`` before anything is launched.  All tensors of a call are on the
current CUDA device.
"""
from __future__ import annotations

import ctypes

# enums of include/iabn_block.h
IABN_Q8_E4M3, IABN_Q8_INT8 = 0, 1
IABN_Q8_GROUP = 128
IABN_NORM_NONE, IABN_NORM_RMS, IABN_NORM_LAYER = 0, 1, 2
IABN_GLU_SILU, IABN_GLU_GELU, IABN_GLU_GELU_TANH = 0, 1, 2
IABN_BLOCK_MAX_COLS = 32768

# Symbols include/iabn_block.h declares.
BLOCK_EXPORTS = ("iabn_checkpoint8_store", "iabn_checkpoint8_load", "iabn_block_norm_forward",
                 "iabn_block_norm_forward_checkpoint8", "iabn_block_norm_workspace_size",
                 "iabn_block_norm_backward", "iabn_block_norm_backward_checkpoint8",
                 "iabn_gated_forward", "iabn_gated_forward_checkpoint8", "iabn_gated_backward",
                 "iabn_gated_backward_checkpoint8")


class IabnBlockDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("rows_per_gate", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("post", ctypes.c_int32), ("pre", ctypes.c_int32), ("format", ctypes.c_int32),
                ("residual_scale", ctypes.c_float), ("eps_post", ctypes.c_float),
                ("eps_pre", ctypes.c_float)]


class IabnGatedDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("ld_grad", ctypes.c_int64), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("format", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of the entry points of a loaded libiabn.so."""
    vp, i32, i64, size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    pb, pg = ctypes.POINTER(IabnBlockDesc), ctypes.POINTER(IabnGatedDesc)
    for name, args in (
            ("iabn_checkpoint8_store", [i64, i64, i64, i32, i32] + [vp] * 4),
            ("iabn_checkpoint8_load", [i64, i64, i64, i32, i32] + [vp] * 6),
            ("iabn_block_norm_forward", [pb] + [vp] * 14),
            ("iabn_block_norm_forward_checkpoint8", [pb] + [vp] * 16),
            ("iabn_block_norm_backward", [pb] + [vp] * 20 + [size, vp]),
            ("iabn_block_norm_backward_checkpoint8", [pb] + [vp] * 20 + [size, vp]),
            ("iabn_gated_forward", [pg] + [vp] * 4),
            ("iabn_gated_forward_checkpoint8", [pg] + [vp] * 8),
            ("iabn_gated_backward", [pg] + [vp] * 7),
            ("iabn_gated_backward_checkpoint8", [pg] + [vp] * 9)):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = i32
    L.iabn_block_norm_workspace_size.argtypes = [pb]
    L.iabn_block_norm_workspace_size.restype = size


# ------------------------------------------------------------------ checks
# A call of a few tokens takes the GPU two to four microseconds, less than an
# ordinary way of checking ten tensors takes the host.  So what a check needs
# is looked up once, when torch is there (_Torch), and each check reads every
# property of a tensor once.

class _Torch:
    """What the calls need of torch and of the package, looked up at the first
    call."""

    def __init__(self):
        import torch
        from . import IABN_ERR_INVALID_ARG, IabnError, lib
        self.float32, self.uint8 = torch.float32, torch.uint8
        self.storage = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        self.formats = {torch.float8_e4m3fn: IABN_Q8_E4M3, torch.int8: IABN_Q8_INT8}
        self.current_device = torch.cuda.current_device
        self.current_stream = torch.cuda.current_stream
        # the current stream of a device without an object around it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.error, self.invalid = IabnError, IABN_ERR_INVALID_ARG
        self.lib = lib()


_torch = None


def _t() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _raise(what: str):
    from . import IABN_ERR_INVALID_ARG, IabnError
    raise IabnError(IABN_ERR_INVALID_ARG, what)


def _rows_of(t, name: str):
    """(rows, cols, row stride) of a [..., cols] tensor whose rows are evenly
    spaced and whose columns are consecutive."""
    shape = t.shape
    if not shape:
        _raise(f"{name} has no columns")
    cols = shape[-1]
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols, cols
    strides = t.stride()
    if strides[-1] != 1 and cols > 1:
        _raise(f"{name}: columns are not consecutive")
    rows, ld = 1, None
    for size, stride in zip(shape[-2::-1], strides[-2::-1]):
        if size != 1:
            if ld is None:
                ld = stride
            elif stride != ld * rows:
                _raise(f"{name}: rows are not evenly spaced")
            rows *= size
    return rows, cols, ld if ld is not None else cols


class _Call:
    """The tensors of one call, checked: all on the current device, of the
    wanted type and number of elements."""

    __slots__ = ("T", "device", "rows", "cols", "numel", "dtype", "storage")

    def __init__(self, first, name: str):
        if first is None:
            _raise(f"{name} is needed")
        device = first.get_device()
        if device < 0:
            _raise(f"{name} is not on a CUDA device")
        self.T = T = _t()
        if device != T.current_device():
            _raise(f"{name} is on device {device}, not on the current one")
        self.device = device
        self.rows, self.cols, _ = _rows_of(first, name)
        self.numel = self.rows * self.cols
        self.dtype = first.dtype
        self.storage = T.storage.get(first.dtype)
        if self.storage is None:
            _raise(f"{name}: unsupported storage dtype {first.dtype}")

    def _refuse(self, t, name: str, dtype, numel: int):
        if t.dtype != dtype:
            _raise(f"{name}: type {t.dtype}, not {dtype}")
        if t.get_device() != self.device:
            _raise(f"{name} is not on the device of the others")
        _raise(f"{name}: {tuple(t.shape)} is not a contiguous tensor of {numel} elements")

    def same(self, t, name: str):
        """A contiguous tensor of the first one's type and rows x cols."""
        if t is None:
            return None
        if t.dtype != self.dtype or t.get_device() != self.device or t.numel() != self.numel \
                or not t.is_contiguous():
            self._refuse(t, name, self.dtype, self.numel)
        shape = t.shape
        if not shape or shape[-1] != self.cols:
            _raise(f"{name}: {tuple(shape)} has not {self.cols} columns")
        return t.data_ptr()

    def floats(self, t, name: str, numel: int):
        """A contiguous float32 tensor of `numel` elements."""
        if t is None:
            return None
        if t.dtype != self.T.float32 or t.get_device() != self.device or t.numel() != numel \
                or not t.is_contiguous():
            self._refuse(t, name, self.T.float32, numel)
        return t.data_ptr()

    def strided(self, t, name: str):
        """(pointer, row stride) of a tensor of the first one's type and size."""
        if t is None:
            _raise(f"{name} is needed")
        if t.dtype != self.dtype or t.get_device() != self.device:
            _raise(f"{name}: type {t.dtype} on {t.device}, not as the others")
        rows, cols, ld = _rows_of(t, name)
        if rows != self.rows or cols != self.cols:
            _raise(f"{name}: {tuple(t.shape)} is not {self.rows} rows of {self.cols}")
        return t.data_ptr(), ld

    def per_col(self, t, name: str):
        return None if t is None else self.floats(t, name, self.cols)

    def per_row(self, t, name: str):
        return None if t is None else self.floats(t, name, self.rows)

    def codes(self, q, scale, name: str, format_of=None):
        """Pointers of codes and scales, and the format."""
        if q is None or scale is None:
            if q is not None or scale is not None:
                _raise(f"{name}: codes and scales go together")
            return None, None, format_of
        form = self.T.formats.get(q.dtype)
        if form is None:
            _raise(f"{name}: codes of type {q.dtype}")
        if format_of is not None and format_of != form:
            _raise(f"{name}: codes of two formats in one call")
        if q.get_device() != self.device or q.numel() != self.numel or not q.is_contiguous():
            self._refuse(q, name, q.dtype, self.numel)
        groups = -(-self.cols // IABN_Q8_GROUP)
        return q.data_ptr(), self.floats(scale, f"scale of {name}", self.rows * groups), form

    def gate(self, t, name: str, rows_per_gate: int):
        if t is None:
            return None
        if not 0 <= rows_per_gate < 1 << 63:   # (more would be cut to 64 bits)
            _raise(f"rows_per_gate = {rows_per_gate}")
        rows = 1 if rows_per_gate == 0 else -(-self.rows // rows_per_gate)
        return self.floats(t, name, rows * self.cols)

    def stream(self, stream) -> int:
        if stream is None:
            if self.T.raw_stream is not None:
                return self.T.raw_stream(self.device)
            stream = self.T.current_stream()
        return stream.cuda_stream

    def done(self, status: int, what: str) -> None:
        if status:
            raise self.T.error(status, what)


def _lib():
    from . import lib
    return lib()


# -------------------------------------------------------------- block norm

def _block(c: _Call, post, pre, rows_per_gate, residual_scale, eps_post, eps_pre, form):
    return IabnBlockDesc(c.rows, c.cols, rows_per_gate, c.storage, post, pre, form or 0,
                         residual_scale, eps_post, eps_pre)


def block_norm_forward(u, h, h_out, n, *, gamma_post=None, beta_post=None, gate=None,
                       gamma_pre=None, beta_pre=None, mean_post=None, rstd_post=None,
                       mean_pre=None, rstd_pre=None, post: int = IABN_NORM_RMS,
                       pre: int = IABN_NORM_RMS, rows_per_gate: int = 0,
                       residual_scale: float = 1.0, eps_post: float = 1e-6,
                       eps_pre: float = 1e-6, stream=None) -> None:
    """h_out = residual_scale*h + gate*(gamma_post*post(u) + beta_post) and
    n = gamma_pre*pre(h_out) + beta_pre.  u None: n from h alone; h_out None or
    n None (pre = IABN_NORM_NONE): not wanted.  Statistics are written where
    given; u and h_out are what ``block_norm_backward`` takes."""
    c = _Call(h, "h")
    d = _block(c, post, pre, rows_per_gate, residual_scale, eps_post, eps_pre, None)
    c.done(c.T.lib.iabn_block_norm_forward(
        ctypes.byref(d), c.same(u, "u"), c.same(h, "h"), c.same(h_out, "h_out"), c.same(n, "n"),
        c.per_col(gamma_post, "gamma_post"), c.per_col(beta_post, "beta_post"),
        c.gate(gate, "gate", rows_per_gate), c.per_col(gamma_pre, "gamma_pre"),
        c.per_col(beta_pre, "beta_pre"), c.per_row(mean_post, "mean_post"),
        c.per_row(rstd_post, "rstd_post"), c.per_row(mean_pre, "mean_pre"),
        c.per_row(rstd_pre, "rstd_pre"), c.stream(stream)), "iabn_block_norm_forward")


def block_norm_forward_checkpoint8(u, h, h_out, n, *, q_post=None, scale_post=None, q_pre=None,
                                   scale_pre=None, rstd_post=None, rstd_pre=None,
                                   gamma_post=None, beta_post=None, gate=None, gamma_pre=None,
                                   beta_pre=None, post: int = IABN_NORM_RMS,
                                   pre: int = IABN_NORM_RMS, rows_per_gate: int = 0,
                                   residual_scale: float = 1.0, eps_post: float = 1e-6,
                                   eps_pre: float = 1e-6, stream=None) -> None:
    """``block_norm_forward``, keeping post(u) and pre(h_out) in 8 bits."""
    c = _Call(h, "h")
    qp, sp, form = c.codes(q_post, scale_post, "q_post")
    qe, se, form = c.codes(q_pre, scale_pre, "q_pre", form)
    d = _block(c, post, pre, rows_per_gate, residual_scale, eps_post, eps_pre, form)
    c.done(c.T.lib.iabn_block_norm_forward_checkpoint8(
        ctypes.byref(d), c.same(u, "u"), c.same(h, "h"), c.same(h_out, "h_out"), c.same(n, "n"),
        c.per_col(gamma_post, "gamma_post"), c.per_col(beta_post, "beta_post"),
        c.gate(gate, "gate", rows_per_gate), c.per_col(gamma_pre, "gamma_pre"),
        c.per_col(beta_pre, "beta_pre"), c.per_row(rstd_post, "rstd_post"),
        c.per_row(rstd_pre, "rstd_pre"), qp, sp, qe, se, c.stream(stream)),
        "iabn_block_norm_forward_checkpoint8")


def block_norm_workspace_size(rows: int, cols: int, rows_per_gate: int = 0) -> int:
    """Bytes of workspace of the block norm's backward calls (0: invalid sizes)."""
    d = IabnBlockDesc(rows, cols, rows_per_gate)
    return int(_lib().iabn_block_norm_workspace_size(ctypes.byref(d)))


def new_block_norm_workspace(rows: int, cols: int, rows_per_gate: int = 0, device=None):
    """A workspace tensor (uint8) for the block norm's backward calls."""
    import torch
    return torch.empty(block_norm_workspace_size(rows, cols, rows_per_gate), dtype=torch.uint8,
                       device=device)


def _workspace(c: _Call, ws):
    if ws is None:
        _raise("workspace is needed")
    if ws.get_device() != c.device or ws.dtype != c.T.uint8 or not ws.is_contiguous():
        _raise("workspace: not a contiguous uint8 tensor on the device of the others")
    return ws.data_ptr(), ws.numel()


def block_norm_backward(u, h_out, dh_out, dn, dh, du, workspace, *, mean_post=None,
                        rstd_post=None, mean_pre=None, rstd_pre=None, gamma_post=None,
                        beta_post=None, gate=None, gamma_pre=None, dgamma_post=None,
                        dbeta_post=None, dgate=None, dgamma_pre=None, dbeta_pre=None,
                        post: int = IABN_NORM_RMS, pre: int = IABN_NORM_RMS,
                        rows_per_gate: int = 0, residual_scale: float = 1.0,
                        stream=None) -> None:
    """Gradients of ``block_norm_forward`` from the kept u and h_out: dh and du
    from dh_out and dn, and those of the parameters that are given."""
    c = _Call(dh, "dh")
    d = _block(c, post, pre, rows_per_gate, residual_scale, 0.0, 0.0, None)
    ws, ws_bytes = _workspace(c, workspace)
    c.done(c.T.lib.iabn_block_norm_backward(
        ctypes.byref(d), c.same(u, "u"), c.same(h_out, "h_out"), c.same(dh_out, "dh_out"),
        c.same(dn, "dn"), c.same(dh, "dh"), c.same(du, "du"), c.per_col(gamma_post, "gamma_post"),
        c.per_col(beta_post, "beta_post"), c.gate(gate, "gate", rows_per_gate),
        c.per_col(gamma_pre, "gamma_pre"), c.per_row(mean_post, "mean_post"),
        c.per_row(rstd_post, "rstd_post"), c.per_row(mean_pre, "mean_pre"),
        c.per_row(rstd_pre, "rstd_pre"), c.per_col(dgamma_post, "dgamma_post"),
        c.per_col(dbeta_post, "dbeta_post"), c.gate(dgate, "dgate", rows_per_gate),
        c.per_col(dgamma_pre, "dgamma_pre"), c.per_col(dbeta_pre, "dbeta_pre"), ws, ws_bytes,
        c.stream(stream)), "iabn_block_norm_backward")


def block_norm_backward_checkpoint8(q_post, q_pre, dh_out, dn, dh, du, workspace, *,
                                    scale_post=None, rstd_post=None, scale_pre=None,
                                    rstd_pre=None, gamma_post=None, beta_post=None, gate=None,
                                    gamma_pre=None, dgamma_post=None, dbeta_post=None,
                                    dgate=None, dgamma_pre=None, dbeta_pre=None,
                                    post: int = IABN_NORM_RMS, pre: int = IABN_NORM_RMS,
                                    rows_per_gate: int = 0, residual_scale: float = 1.0,
                                    stream=None) -> None:
    """``block_norm_backward`` from the 8-bit checkpoints."""
    c = _Call(dh, "dh")
    qp, sp, form = c.codes(q_post, scale_post, "q_post")
    qe, se, form = c.codes(q_pre, scale_pre, "q_pre", form)
    d = _block(c, post, pre, rows_per_gate, residual_scale, 0.0, 0.0, form)
    ws, ws_bytes = _workspace(c, workspace)
    c.done(c.T.lib.iabn_block_norm_backward_checkpoint8(
        ctypes.byref(d), qp, sp, qe, se, c.same(dh_out, "dh_out"), c.same(dn, "dn"),
        c.same(dh, "dh"), c.same(du, "du"), c.per_col(gamma_post, "gamma_post"),
        c.per_col(beta_post, "beta_post"), c.gate(gate, "gate", rows_per_gate),
        c.per_col(gamma_pre, "gamma_pre"), c.per_row(rstd_post, "rstd_post"),
        c.per_row(rstd_pre, "rstd_pre"), c.per_col(dgamma_post, "dgamma_post"),
        c.per_col(dbeta_post, "dbeta_post"), c.gate(dgate, "dgate", rows_per_gate),
        c.per_col(dgamma_pre, "dgamma_pre"), c.per_col(dbeta_pre, "dbeta_pre"), ws, ws_bytes,
        c.stream(stream)), "iabn_block_norm_backward_checkpoint8")


# -------------------------------------------------------- gated activation

def _pair(c: _Call, a, b, names: str):
    pa, ld = c.strided(a, names[0])
    pb, ldb = c.strided(b, names[1])
    if ld != ldb:
        _raise(f"{names[0]} and {names[1]} have different row strides")
    return pa, pb, ld


def gated_forward(a, b, z, *, act: int = IABN_GLU_SILU, stream=None) -> None:
    """z = phi(a)*b."""
    c = _Call(z, "z")
    pa, pb, ld = _pair(c, a, b, ("a", "b"))
    d = IabnGatedDesc(c.rows, c.cols, ld, c.cols, c.storage, act, 0)
    c.done(c.T.lib.iabn_gated_forward(ctypes.byref(d), pa, pb, c.same(z, "z"), c.stream(stream)),
          "iabn_gated_forward")


def gated_forward_checkpoint8(a, b, z, qa, scale_a, qb, scale_b, *, act: int = IABN_GLU_SILU,
                              stream=None) -> None:
    """z = phi(a)*b, keeping a and b in 8 bits."""
    c = _Call(z, "z")
    pa, pb, ld = _pair(c, a, b, ("a", "b"))
    ca, sa, form = c.codes(qa, scale_a, "qa")
    cb, sb, form = c.codes(qb, scale_b, "qb", form)
    d = IabnGatedDesc(c.rows, c.cols, ld, c.cols, c.storage, act, form or 0)
    c.done(c.T.lib.iabn_gated_forward_checkpoint8(ctypes.byref(d), pa, pb, c.same(z, "z"), ca, sa,
                                                cb, sb, c.stream(stream)),
          "iabn_gated_forward_checkpoint8")


def gated_backward(a, b, dz, da, db, *, z=None, act: int = IABN_GLU_SILU, stream=None) -> None:
    """da and db from dz and the kept a and b; z again where it is given."""
    c = _Call(dz, "dz")
    pa, pb, ld = _pair(c, a, b, ("a", "b"))
    pda, pdb, ld_grad = _pair(c, da, db, ("da", "db"))
    d = IabnGatedDesc(c.rows, c.cols, ld, ld_grad, c.storage, act, 0)
    c.done(c.T.lib.iabn_gated_backward(ctypes.byref(d), pa, pb, c.same(dz, "dz"), pda, pdb,
                                     c.same(z, "z"), c.stream(stream)), "iabn_gated_backward")


def gated_backward_checkpoint8(qa, scale_a, qb, scale_b, dz, da, db, *, z=None,
                               act: int = IABN_GLU_SILU, stream=None) -> None:
    """``gated_backward`` from the 8-bit checkpoints."""
    c = _Call(dz, "dz")
    pda, pdb, ld_grad = _pair(c, da, db, ("da", "db"))
    ca, sa, form = c.codes(qa, scale_a, "qa")
    cb, sb, form = c.codes(qb, scale_b, "qb", form)
    d = IabnGatedDesc(c.rows, c.cols, c.cols, ld_grad, c.storage, act, form or 0)
    c.done(c.T.lib.iabn_gated_backward_checkpoint8(ctypes.byref(d), ca, sa, cb, sb,
                                                 c.same(dz, "dz"), pda, pdb, c.same(z, "z"),
                                                 c.stream(stream)),
          "iabn_gated_backward_checkpoint8")


# ------------------------------------------------------- 8-bit checkpoints

def checkpoint8_store(x, q, scale, *, stream=None) -> None:
    """Keeps x in 8 bits: q and scale are written."""
    c = _Call(x, "x")
    px, ld = c.strided(x, "x")
    pq, ps, form = c.codes(q, scale, "q")
    c.done(c.T.lib.iabn_checkpoint8_store(c.rows, c.cols, ld, c.storage, form or 0, px, pq, ps,
                                        c.stream(stream)), "iabn_checkpoint8_store")


def checkpoint8_load(q, scale, y, *, gamma=None, beta=None, stream=None) -> None:
    """y = gamma*value + beta of the kept values."""
    c = _Call(y, "y")
    py, ld = c.strided(y, "y")
    pq, ps, form = c.codes(q, scale, "q")
    c.done(c.T.lib.iabn_checkpoint8_load(c.rows, c.cols, ld, c.storage, form or 0, pq, ps,
                                       c.per_col(gamma, "gamma"), c.per_col(beta, "beta"), py,
                                       c.stream(stream)), "iabn_checkpoint8_load")
