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

from . import GC_OK, GCError, lib

GC_F32, GC_BF16, GC_F16 = 0, 1, 2
GC_ACCUMULATE = 0x1
GC_GATE_SILU, GC_GATE_GELU_TANH = 0, 1
ACT_GROUP = 32

_DTYPES = {torch.float32: GC_F32, torch.bfloat16: GC_BF16, torch.float16: GC_F16}


_current = torch._C._cuda_getCurrentRawStream      # torch.cuda.current_stream() builds an object around it


def _bad(what):
    raise ValueError(what)


def _check(status, what):
    if status != GC_OK:
        raise GCError(status, what)


def _stream(stream, device):
    """The cudaStream_t of a torch stream or of a number; the current one of
    the device for None."""
    if stream is None:
        return _current(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _mat(t, name, rows=None, cols=None, dtype=None):
    """(pointer, row stride) of a matrix argument, after its checks."""
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda:
        _bad(f"{name}: a 2-D CUDA tensor is needed")
    r, c = shape
    if rows is not None and (r != rows or c != cols):
        _bad(f"{name}: shape {(r, c)} where {(rows, cols)} is needed")
    if dtype is not None and t.dtype is not dtype:
        _bad(f"{name}: {t.dtype} where {dtype} is needed")
    s0, s1 = t.stride()
    if s1 != 1 and c > 1:
        _bad(f"{name}: columns are not consecutive")
    if s0 < c:
        if r > 1:
            _bad(f"{name}: rows overlap")
        s0 = c
    return t.data_ptr(), s0


def _vec(t, name, n, dtypes):
    """Pointer of a contiguous vector argument."""
    if t.shape != (n,) or not t.is_cuda or t.dtype not in dtypes or not t.is_contiguous():
        _bad(f"{name}: a contiguous CUDA vector of {n} elements of {' or '.join(str(d) for d in dtypes)} is needed")
    return t.data_ptr()


def _workspace_args(ws, name):
    if not ws.is_cuda or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        _bad(f"{name}: a contiguous CUDA uint8 tensor is needed")
    return ws.data_ptr(), ws.numel()


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
    """(codes, steps) pointers of a checkpoint argument."""
    if ckpt.rows != rows or ckpt.cols != cols:
        _bad(f"{name}: a checkpoint of {(ckpt.rows, ckpt.cols)} where {(rows, cols)} is needed")
    return ckpt._codes, ckpt._steps


def _type(t, name):
    d = _DTYPES.get(t.dtype)
    return _bad(f"{name}: {t.dtype} is not supported") if d is None else d


def act_compress(x, ckpt, stream=None):
    """Writes the checkpoint of x."""
    p, ld = _mat(x, "x", ckpt.rows, ckpt.cols)
    _check(lib().gc_act_compress(p, ld, _type(x, "x"), ckpt.rows, ckpt.cols, ckpt._codes, ckpt._steps,
                                 _stream(stream, x.get_device())), "gc_act_compress")


def act_decompress(ckpt, out, stream=None):
    """Reads a checkpoint back into out, in out's type."""
    p, ld = _mat(out, "out", ckpt.rows, ckpt.cols)
    _check(lib().gc_act_decompress(ckpt._codes, ckpt._steps, ckpt.rows, ckpt.cols, p, ld, _type(out, "out"),
                                   _stream(stream, out.get_device())), "gc_act_decompress")


def rmsnorm(x, weight, eps, y, residual=None, h=None, rstd=None, ckpt=None, stream=None):
    """y = rmsnorm(x + residual) * weight; h = x + residual, rstd and the
    checkpoint of the normalised rows where given.  weight or y may be None."""
    px, ldx = _mat(x, "x")
    rows, cols = x.shape
    dtype = x.dtype
    kind = _type(x, "x")
    pr = ldr = py = ldy = ph = ldh = pw = codes = steps = ps = None
    wkind = 0
    if residual is not None:
        pr, ldr = _mat(residual, "residual", rows, cols, dtype)
    if y is not None:
        py, ldy = _mat(y, "y", rows, cols, dtype)
    if h is not None:
        ph, ldh = _mat(h, "h", rows, cols, dtype)
    if weight is not None:
        pw, wkind = _vec(weight, "weight", cols, _WEIGHTS), _DTYPES[weight.dtype]
    if rstd is not None:
        ps = _vec(rstd, "rstd", rows, _F32)
    if ckpt is not None:
        codes, steps = _held(ckpt, "ckpt", rows, cols)
    _check(lib().gc_rmsnorm(px, ldx, pr, ldr or 0, kind, pw, wkind, eps, rows, cols, py, ldy or 0, ph, ldh or 0, ps,
                            codes, steps, _stream(stream, x.get_device())), "gc_rmsnorm")


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
    dtype = dy.dtype
    pdx, lddx = _mat(dx, "dx", rows, cols, dtype)
    pdh = lddh = pw = pdw = ws = None
    size = wkind = 0
    if dh is not None:
        pdh, lddh = _mat(dh, "dh", rows, cols, dtype)
    if weight is not None:
        pw, wkind = _vec(weight, "weight", cols, _WEIGHTS), _DTYPES[weight.dtype]
    if dw is not None:
        pdw = _vec(dw, "dw", cols, _F32)
        ws, size = _workspace_args(workspace, "workspace") if workspace is not None else (None, 0)
    if rstd is None:
        _bad("rstd is needed")
    _check(lib().gc_rmsnorm_backward(pdy, lddy, pdh, lddh or 0, _type(dy, "dy"), ckpt._codes, ckpt._steps,
                                     _vec(rstd, "rstd", rows, _F32), pw, wkind, rows, cols, pdx, lddx, pdw,
                                     GC_ACCUMULATE if accumulate else 0, ws, size, _stream(stream, dy.get_device())),
           "gc_rmsnorm_backward")


def gated_act(kind, gate, up, out, ckpt_gate=None, ckpt_up=None, stream=None):
    """out = act(gate) * up; the checkpoints of gate and up where given."""
    pg, ldg = _mat(gate, "gate")
    rows, cols = gate.shape
    dtype = gate.dtype
    pu, ldu = _mat(up, "up", rows, cols, dtype)
    po, ldo = _mat(out, "out", rows, cols, dtype)
    gcode = gstep = ucode = ustep = None
    if ckpt_gate is not None:
        gcode, gstep = _held(ckpt_gate, "ckpt_gate", rows, cols)
    if ckpt_up is not None:
        ucode, ustep = _held(ckpt_up, "ckpt_up", rows, cols)
    _check(lib().gc_gated_act(kind, pg, ldg, pu, ldu, _type(gate, "gate"), rows, cols, po, ldo, gcode, gstep, ucode,
                              ustep, _stream(stream, gate.get_device())), "gc_gated_act")


def gated_act_backward(kind, dout, ckpt_gate, ckpt_up, dgate, dup, ckpt_out=None, stream=None):
    """Gradients of gated_act from its checkpoints, and the checkpoint of
    act(gate) * up again where ckpt_out is given."""
    rows, cols = ckpt_gate.rows, ckpt_gate.cols
    pd, ldd = _mat(dout, "dout", rows, cols)
    dtype = dout.dtype
    pg, ldg = _mat(dgate, "dgate", rows, cols, dtype)
    pu, ldu = _mat(dup, "dup", rows, cols, dtype)
    ucode, ustep = _held(ckpt_up, "ckpt_up", rows, cols)
    ocode = ostep = None
    if ckpt_out is not None:
        ocode, ostep = _held(ckpt_out, "ckpt_out", rows, cols)
    _check(lib().gc_gated_act_backward(kind, pd, ldd, _type(dout, "dout"), ckpt_gate._codes, ckpt_gate._steps, ucode,
                                       ustep, rows, cols, pg, ldg, pu, ldu, ocode, ostep,
                                       _stream(stream, dout.get_device())), "gc_gated_act_backward")


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
    n = dy.shape[-1]
    pdy, lddy = _mat(dy, "dy", rows, n)
    pdw, lddw = _mat(dw, "dw", n, k, torch.float32)
    ps, skind = None, 0
    if col_scale is not None:
        ps, skind = _vec(col_scale, "col_scale", k, _WEIGHTS), _DTYPES[col_scale.dtype]
    ws, size = _workspace_args(workspace, "workspace")
    _check(lib().gc_act_weight_grad(pdy, lddy, _type(dy, "dy"), rows, n, ckpt._codes, ckpt._steps, k, ps, skind, pdw,
                                    lddw, GC_ACCUMULATE if accumulate else 0, ws, size,
                                    _stream(stream, dy.get_device())), "gc_act_weight_grad")
