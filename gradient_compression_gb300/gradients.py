"""The global gradient norm over many tensors, and clipping by it.

The gc_grad_* entry points of include/gc.h.  Gradients are given as a list of
dense CUDA tensors of any shapes, fp32, bf16 or fp16 mixed, wherever they lie
at the call (an arena is a list of one): nothing is kept from call to call.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import activations as _act
from . import lib


def grad_norm_workspace(tensors, device=None) -> torch.Tensor:
    """For grad_norm of so many tensors, or fewer; on their GPU unless said."""
    out = C.c_size_t(0)
    _act._check(lib().gc_grad_norm_workspace_size(len(tensors), C.byref(out)), "gc_grad_norm_workspace_size")
    return _act._workspace(out, device or (tensors[0].device if len(tensors) else "cuda"))


def grad_norm(tensors, norm, workspace, stream=None):
    """norm[0] (fp32) = the L2 norm of all elements of all tensors."""
    st = (_act._calls or _act._marshal()).grad_norm(tensors, norm, workspace, stream)
    if st:
        _act._check(st, "gc_grad_norm")


def grad_clip(tensors, norm, max_norm, out=None, stream=None):
    """Every tensor times max_norm / norm[0] where the norm is larger, else as it
    is: in place, or into the tensors of `out` (views of the arena, say), of the
    same shapes or, contiguous, sizes and of any of the types."""
    st = (_act._calls or _act._marshal()).grad_clip(tensors, norm, max_norm, out, stream)
    if st:
        _act._check(st, "gc_grad_clip")
