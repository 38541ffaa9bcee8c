"""8-bit activation checkpoints and the operators that write and read them.

Argument marshalling for the gc_act_* / gc_rmsnorm* / gc_gated_act* entry
points of include/gc.h, which define the results.  Matrices are 2-D CUDA
tensors (fp32, bf16 or fp16) whose columns are consecutive; their row stride
is free, so halves of one projection or slices of a batch need no copy.
Outputs and workspaces are the caller's.  A wrong shape, type or device
raises ValueError before anything is enqueued.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _check, _ptr, _stream, lib

GC_F32, GC_BF16, GC_F16 = 0, 1, 2
GC_ACCUMULATE = 0x1
GC_GATE_SILU, GC_GATE_GELU_TANH = 0, 1
ACT_GROUP = 32

_DTYPES = {torch.float32: GC_F32, torch.bfloat16: GC_BF16, torch.float16: GC_F16}


def _bad(what):
    raise ValueError(what)


def _mat(t, name, rows=None, cols=None, dtype=None):
    """(pointer, row stride) of a matrix argument, after its checks."""
    if t.dim() != 2 or not t.is_cuda:
        _bad(f"{name}: a 2-D CUDA tensor is needed")
    r, c = t.shape
    if rows is not None and (r != rows or c != cols):
        _bad(f"{name}: shape {(r, c)} where {(rows, cols)} is needed")
    if dtype is not None and t.dtype is not dtype:
        _bad(f"{name}: {t.dtype} where {dtype} is needed")
    s0, s1 = t.stride()
    if s1 != 1 and c > 1:
        _bad(f"{name}: columns are not consecutive")
    if r <= 1:
        s0 = max(c, 1)
    elif s0 < c:
        _bad(f"{name}: rows overlap")
    return t.data_ptr(), s0


def _opt(t, name, rows, cols, dtype):
    return (None, 0) if t is None else _mat(t, name, rows, cols, dtype)


def _vec(t, name, n, dtypes):
    """Pointer of a contiguous vector argument; None stays None."""
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != n or not t.is_cuda or t.dtype not in dtypes or (n > 1 and t.stride(0) != 1):
        _bad(f"{name}: a contiguous CUDA vector of {n} elements of {' or '.join(str(d) for d in dtypes)} is needed")
    return t.data_ptr()


def _dtype(t, name):
    d = _DTYPES.get(t.dtype)
    return _bad(f"{name}: {t.dtype} is not supported") if d is None else d


_F32 = (torch.float32,)
_WEIGHTS = tuple(_DTYPES)


class ActCheckpoint:
    """Codes and steps of an activation x[rows, cols] held in 8 bits.

    codes int8[rows, ldc] with ldc = 32 * ceil(cols / 32), steps uint8[rows,
    ldc / 32]; allocated here unless given."""

    __slots__ = ("rows", "cols", "codes", "steps", "_codes", "_steps")

    def __init__(self, rows, cols, device="cuda", codes=None, steps=None):
        self.rows, self.cols = int(rows), int(cols)
        if self.rows < 0 or self.cols < 1:
            _bad(f"a checkpoint of {rows} x {cols}")
        groups = (self.cols + ACT_GROUP - 1) // ACT_GROUP
        shape = (self.rows, groups * ACT_GROUP)
        if codes is None:
            codes = torch.empty(shape, dtype=torch.int8, device=device)
        if steps is None:
            steps = torch.empty((self.rows, groups), dtype=torch.uint8, device=device)
        if codes.shape != shape or codes.dtype is not torch.int8 or not codes.is_contiguous() or not codes.is_cuda:
            _bad(f"codes: a contiguous CUDA int8 tensor of shape {shape} is needed")
        if steps.shape != (self.rows, groups) or steps.dtype is not torch.uint8 or not steps.is_contiguous() \
                or not steps.is_cuda:
            _bad(f"steps: a contiguous CUDA uint8 tensor of shape {(self.rows, groups)} is needed")
        self.codes, self.steps = codes, steps
        self._codes, self._steps = codes.data_ptr(), steps.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.steps.numel()


def _held(ckpt, name, rows, cols):
    """(codes, steps) pointers of a checkpoint argument; None stays None."""
    if ckpt is None:
        return None, None
    if ckpt.rows != rows or ckpt.cols != cols:
        _bad(f"{name}: a checkpoint of {(ckpt.rows, ckpt.cols)} where {(rows, cols)} is needed")
    return ckpt._codes, ckpt._steps


def act_compress(x, ckpt, stream=None):
    """Writes the checkpoint of x."""
    p, ld = _mat(x, "x", ckpt.rows, ckpt.cols)
    _check(lib().gc_act_compress(p, ld, _dtype(x, "x"), ckpt.rows, ckpt.cols, ckpt._codes, ckpt._steps,
                                 _stream(stream)), "gc_act_compress")


def act_decompress(ckpt, out, stream=None):
    """Reads a checkpoint back into out, in out's type."""
    p, ld = _mat(out, "out", ckpt.rows, ckpt.cols)
    _check(lib().gc_act_decompress(ckpt._codes, ckpt._steps, ckpt.rows, ckpt.cols, p, ld, _dtype(out, "out"),
                                   _stream(stream)), "gc_act_decompress")


def rmsnorm(x, weight, eps, y, residual=None, h=None, rstd=None, ckpt=None, stream=None):
    """y = rmsnorm(x + residual) * weight; h = x + residual, rstd and the
    checkpoint of the normalised rows where given.  weight or y may be None."""
    rows, cols = x.shape if x.dim() == 2 else _bad("x: a 2-D CUDA tensor is needed")
    px, ldx = _mat(x, "x")
    pr, ldr = _opt(residual, "residual", rows, cols, x.dtype)
    py, ldy = _opt(y, "y", rows, cols, x.dtype)
    ph, ldh = _opt(h, "h", rows, cols, x.dtype)
    pw = _vec(weight, "weight", cols, _WEIGHTS)
    codes, steps = _held(ckpt, "ckpt", rows, cols)
    _check(lib().gc_rmsnorm(px, ldx, pr, ldr, _dtype(x, "x"), pw, 0 if weight is None else _DTYPES[weight.dtype],
                            eps, rows, cols, py, ldy, ph, ldh, _vec(rstd, "rstd", rows, _F32), codes, steps,
                            _stream(stream)), "gc_rmsnorm")


def _workspace(size, device):
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(size.value), 256), dtype=torch.uint8, device=device)


def rmsnorm_backward_workspace(rows, cols, device="cuda") -> torch.Tensor:
    out = C.c_size_t(0)
    _check(lib().gc_rmsnorm_backward_workspace_size(int(rows), int(cols), C.byref(out)),
           "gc_rmsnorm_backward_workspace_size")
    return _workspace(out, device)


def rmsnorm_backward(dy, ckpt, rstd, weight, dx, dw, workspace, dh=None, accumulate=False, stream=None):
    """Gradients of rmsnorm from its checkpoint: dx (of x and of the residual,
    the gradient dh that arrives at h added), dw fp32[cols].  weight, dw (and
    then workspace) may be None."""
    rows, cols = ckpt.rows, ckpt.cols
    pdy, lddy = _mat(dy, "dy", rows, cols)
    pdh, lddh = _opt(dh, "dh", rows, cols, dy.dtype)
    pdx, lddx = _mat(dx, "dx", rows, cols, dy.dtype)
    pw = _vec(weight, "weight", cols, _WEIGHTS)
    if rstd is None:
        _bad("rstd is needed")
    _check(lib().gc_rmsnorm_backward(pdy, lddy, pdh, lddh, _dtype(dy, "dy"), ckpt._codes, ckpt._steps,
                                     _vec(rstd, "rstd", rows, _F32), pw,
                                     0 if weight is None else _DTYPES[weight.dtype], rows, cols, pdx, lddx,
                                     _vec(dw, "dw", cols, _F32), GC_ACCUMULATE if accumulate else 0, _ptr(workspace),
                                     0 if workspace is None else workspace.numel(), _stream(stream)),
           "gc_rmsnorm_backward")


def gated_act(kind, gate, up, out, ckpt_gate=None, ckpt_up=None, stream=None):
    """out = act(gate) * up; the checkpoints of gate and up where given."""
    rows, cols = gate.shape if gate.dim() == 2 else _bad("gate: a 2-D CUDA tensor is needed")
    pg, ldg = _mat(gate, "gate")
    pu, ldu = _mat(up, "up", rows, cols, gate.dtype)
    po, ldo = _mat(out, "out", rows, cols, gate.dtype)
    gc_, gs = _held(ckpt_gate, "ckpt_gate", rows, cols)
    uc, us = _held(ckpt_up, "ckpt_up", rows, cols)
    _check(lib().gc_gated_act(kind, pg, ldg, pu, ldu, _dtype(gate, "gate"), rows, cols, po, ldo, gc_, gs, uc, us,
                              _stream(stream)), "gc_gated_act")


def gated_act_backward(kind, dout, ckpt_gate, ckpt_up, dgate, dup, ckpt_out=None, stream=None):
    """Gradients of gated_act from its checkpoints, and the checkpoint of
    act(gate) * up again where ckpt_out is given."""
    rows, cols = ckpt_gate.rows, ckpt_gate.cols
    pd, ldd = _mat(dout, "dout", rows, cols)
    pg, ldg = _mat(dgate, "dgate", rows, cols, dout.dtype)
    pu, ldu = _mat(dup, "dup", rows, cols, dout.dtype)
    uc, us = _held(ckpt_up, "ckpt_up", rows, cols)
    oc, os_ = _held(ckpt_out, "ckpt_out", rows, cols)
    _check(lib().gc_gated_act_backward(kind, pd, ldd, _dtype(dout, "dout"), ckpt_gate._codes, ckpt_gate._steps, uc,
                                       us, rows, cols, pg, ldg, pu, ldu, oc, os_, _stream(stream)),
           "gc_gated_act_backward")


def act_weight_grad_workspace(rows, n, k, dtype, device="cuda") -> torch.Tensor:
    out = C.c_size_t(0)
    if dtype not in _DTYPES:
        _bad(f"{dtype} is not supported")
    _check(lib().gc_act_weight_grad_workspace_size(int(rows), int(n), int(k), _DTYPES[dtype], C.byref(out)),
           "gc_act_weight_grad_workspace_size")
    return _workspace(out, device)


def act_weight_grad(dy, ckpt, dw, workspace, col_scale=None, accumulate=False, stream=None):
    """dw[n, k] = (dw +) col_scale[k] * sum over rows of dy[rows, n] * x[rows, k]
    with x the checkpoint's values; dw is fp32, e.g. a view of the arena."""
    rows, k = ckpt.rows, ckpt.cols
    n = dy.shape[1] if dy.dim() == 2 else _bad("dy: a 2-D CUDA tensor is needed")
    pdy, lddy = _mat(dy, "dy", rows, n)
    pdw, lddw = _mat(dw, "dw", n, k, torch.float32)
    ps = _vec(col_scale, "col_scale", k, _WEIGHTS)
    _check(lib().gc_act_weight_grad(pdy, lddy, _dtype(dy, "dy"), rows, n, ckpt._codes, ckpt._steps, k, ps,
                                    0 if col_scale is None else _DTYPES[col_scale.dtype], pdw, lddw,
                                    GC_ACCUMULATE if accumulate else 0, _ptr(workspace), workspace.numel(),
                                    _stream(stream)), "gc_act_weight_grad")
