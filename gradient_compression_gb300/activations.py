"""8-bit activation checkpoints and the operators that write and read them.

The gc_act_* / gc_rmsnorm* / gc_gated_act* entry points of include/gc.h, which
define the results.  Matrices are 2-D CUDA tensors (fp32, bf16 or fp16) whose
columns are consecutive; their row stride is free, so halves of one projection
or slices of a batch need no copy.  Outputs and workspaces are the caller's.
A wrong shape, type or device raises ValueError before anything is enqueued;
the checks and the calls are compiled (csrc/gc_marshal.cpp), since calls of a
few tokens cost little else.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import GC_OK, GCError, lib

GC_F32, GC_BF16, GC_F16 = 0, 1, 2
GC_ACCUMULATE = 0x1
GC_COPY_ROWS, GC_COPY_WEIGHTS = 0x1, 0x2
GC_GATE_SILU, GC_GATE_GELU_TANH = 0, 1
ACT_GROUP = 32

_DTYPES = {torch.float32: GC_F32, torch.bfloat16: GC_BF16, torch.float16: GC_F16}

_calls = None


def _marshal():
    """The compiled calls, bound to libgc's entry points."""
    global _calls
    L = lib()
    from . import _marshal as m
    names = ("act_compress", "act_decompress", "rmsnorm", "rmsnorm_backward", "gated_act", "gated_act_backward",
             "act_weight_grad", "gated_proj", "gated_proj_backward", "grad_norm", "grad_clip")
    m.bind(*(C.cast(getattr(L, "gc_" + n), C.c_void_p).value for n in names))
    _calls = m
    return m


def _bad(what):
    raise ValueError(what)


def _check(status, what):
    if status != GC_OK:
        raise GCError(status, what)


class ActCheckpoint:
    """Codes and steps of an activation x[rows, cols] held in 8 bits.

    codes int8[rows, ldc] with ldc = 32 * ceil(cols / 32), steps uint8[rows,
    ldc / 32]; allocated here unless given.  Every call takes the two tensors
    as they are then, so they may be moved away and put back."""

    __slots__ = ("rows", "cols", "codes", "steps")

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
        (_calls or _marshal()).checkpoint(codes, steps, self.rows, self.cols)
        self.codes, self.steps = codes, steps

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.steps.numel()


def act_compress(x, ckpt, stream=None):
    """Writes the checkpoint of x."""
    st = (_calls or _marshal()).act_compress(x, ckpt, stream)
    if st:
        _check(st, "gc_act_compress")


def act_decompress(ckpt, out, stream=None):
    """Reads a checkpoint back into out, in out's type."""
    st = (_calls or _marshal()).act_decompress(ckpt, out, stream)
    if st:
        _check(st, "gc_act_decompress")


def rmsnorm(x, weight, eps, y, residual=None, h=None, rstd=None, ckpt=None, stream=None):
    """y = rmsnorm(x + residual) * weight; h = x + residual, rstd and the
    checkpoint of the normalised rows where given.  weight or y may be None."""
    st = (_calls or _marshal()).rmsnorm(x, weight, eps, y, residual, h, rstd, ckpt, stream)
    if st:
        _check(st, "gc_rmsnorm")


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
    st = (_calls or _marshal()).rmsnorm_backward(dy, ckpt, rstd, weight, dx, dw, workspace, dh, accumulate, stream)
    if st:
        _check(st, "gc_rmsnorm_backward")


def gated_act(kind, gate, up, out, ckpt_gate=None, ckpt_up=None, stream=None):
    """out = act(gate) * up; the checkpoints of gate and up where given."""
    st = (_calls or _marshal()).gated_act(kind, gate, up, out, ckpt_gate, ckpt_up, stream)
    if st:
        _check(st, "gc_gated_act")


def gated_act_backward(kind, dout, ckpt_gate, ckpt_up, dgate, dup, ckpt_out=None, stream=None):
    """Gradients of gated_act from its checkpoints, and the checkpoint of
    act(gate) * up again where ckpt_out is given."""
    st = (_calls or _marshal()).gated_act_backward(kind, dout, ckpt_gate, ckpt_up, dgate, dup, ckpt_out, stream)
    if st:
        _check(st, "gc_gated_act_backward")


def _unaligned(*mats):
    """Whether one of the matrices does not start its rows on 16-byte boundaries."""
    return any(t.data_ptr() % 16 or max(t.stride(0), t.size(1)) * t.element_size() % 16 for t in mats)


def _gated_proj_workspace(entry, rows, w_gate, w_up):
    for t in (*rows, w_gate, w_up):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            _bad("2-D tensors are needed")
    out = C.c_size_t(0)
    copied = (GC_COPY_ROWS if _unaligned(*rows) else 0) | (GC_COPY_WEIGHTS if _unaligned(w_gate, w_up) else 0)
    _check(getattr(lib(), entry)(rows[0].size(0), w_gate.size(0), w_gate.size(1), copied, C.byref(out)), entry)
    return _workspace(out, w_gate.device)


def gated_proj_workspace(x, w_gate, w_up) -> torch.Tensor:
    """For gated_proj of these, or of others of the same sizes, or fewer rows,
    that need as few copies (those whose rows do not start on 16-byte boundaries)."""
    return _gated_proj_workspace("gc_gated_proj_workspace_size", (x,), w_gate, w_up)


def gated_proj(kind, x, w_gate, w_up, out, workspace, ckpt_gate=None, ckpt_up=None, stream=None):
    """out[rows, n] = act(x @ w_gate.T) * (x @ w_up.T), and the checkpoints of the
    two products where given; x[rows, k], weights [n, k], bf16 or fp16."""
    st = (_calls or _marshal()).gated_proj(kind, x, w_gate, w_up, out, workspace, ckpt_gate, ckpt_up, stream)
    if st:
        _check(st, "gc_gated_proj")


def gated_proj_backward_workspace(dgate, dup, w_gate, w_up) -> torch.Tensor:
    """For gated_proj_backward, as gated_proj_workspace is for gated_proj."""
    return _gated_proj_workspace("gc_gated_proj_backward_workspace_size", (dgate, dup), w_gate, w_up)


def gated_proj_backward(kind, dout, ckpt_gate, ckpt_up, w_gate, w_up, dgate, dup, dx, workspace, ckpt_out=None,
                        stream=None):
    """Gradients of gated_proj from its checkpoints: dgate and dup (and the
    checkpoint of act(gate) * up again) as gated_act_backward gives them, and
    dx = dgate @ w_gate + dup @ w_up.  The weights' come from act_weight_grad."""
    st = (_calls or _marshal()).gated_proj_backward(kind, dout, ckpt_gate, ckpt_up, w_gate, w_up, dgate, dup, dx,
                                                    workspace, ckpt_out, stream)
    if st:
        _check(st, "gc_gated_proj_backward")


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
    st = (_calls or _marshal()).act_weight_grad(dy, ckpt, dw, workspace, col_scale, accumulate, stream)
    if st:
        _check(st, "gc_act_weight_grad")
