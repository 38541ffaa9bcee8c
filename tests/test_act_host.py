"""Activation-checkpoint entry points: arguments refused on the host before
anything is enqueued (CPU only)."""
import ctypes as C

import pytest
import torch

A = 0x10000          # stands for an aligned device address; no call below gets as far as using it


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    gcmod.lib()
    return gcmod


def test_compress_refusals(gc):
    f = gc.lib().gc_act_compress
    assert f(A, 64, gc.GC_BF16, -1, 64, A, A, None) == gc.GC_ERR_LAYOUT
    assert f(A, 64, gc.GC_BF16, 4, 0, A, A, None) == gc.GC_ERR_LAYOUT
    assert f(A, 63, gc.GC_BF16, 4, 64, A, A, None) == gc.GC_ERR_LAYOUT
    assert f(A, 64, gc.GC_BF16, 1 << 31, 64, A, A, None) == gc.GC_ERR_LAYOUT
    assert f(A, 64, 3, 4, 64, A, A, None) == gc.GC_ERR_INVALID_ARG
    assert f(None, 64, gc.GC_F32, 4, 64, A, A, None) == gc.GC_ERR_INVALID_ARG
    assert f(A, 64, gc.GC_F32, 4, 64, None, A, None) == gc.GC_ERR_INVALID_ARG
    assert f(A, 64, gc.GC_F32, 4, 64, A, None, None) == gc.GC_ERR_INVALID_ARG
    assert f(A + 2, 64, gc.GC_F32, 4, 64, A, A, None) == gc.GC_ERR_ALIGNMENT
    assert f(A, 64, gc.GC_F32, 4, 64, A + 8, A, None) == gc.GC_ERR_ALIGNMENT
    assert f(None, 64, gc.GC_F32, 0, 64, None, None, None) == gc.GC_OK          # no rows: nothing to do


def test_decompress_refusals(gc):
    f = gc.lib().gc_act_decompress
    assert f(A, A, 4, 64, A, 63, gc.GC_F16, None) == gc.GC_ERR_LAYOUT
    assert f(A, A, 4, 64, None, 64, gc.GC_F16, None) == gc.GC_ERR_INVALID_ARG
    assert f(A, A, 4, 64, A, 64, -1, None) == gc.GC_ERR_INVALID_ARG
    assert f(A + 1, A, 4, 64, A, 64, gc.GC_F16, None) == gc.GC_ERR_ALIGNMENT
    assert f(None, None, 0, 64, None, 64, gc.GC_F16, None) == gc.GC_OK


def test_rmsnorm_refusals(gc):
    def f(x=A, ldx=64, r=None, ldr=0, dt=1, w=A, wt=1, eps=1e-5, rows=4, cols=64, y=A, ldy=64, h=None, ldh=0,
          rstd=None, codes=None, steps=None):
        return gc.lib().gc_rmsnorm(x, ldx, r, ldr, dt, w, wt, eps, rows, cols, y, ldy, h, ldh, rstd, codes, steps, None)

    assert f(eps=-1e-6) == gc.GC_ERR_INVALID_ARG
    assert f(eps=float("nan")) == gc.GC_ERR_INVALID_ARG
    assert f(wt=7) == gc.GC_ERR_INVALID_ARG
    assert f(x=None) == gc.GC_ERR_INVALID_ARG
    assert f(r=A, ldr=63) == gc.GC_ERR_LAYOUT
    assert f(h=A, ldh=1) == gc.GC_ERR_LAYOUT
    assert f(y=A + 1) == gc.GC_ERR_ALIGNMENT
    assert f(codes=A) == gc.GC_ERR_INVALID_ARG          # a checkpoint is codes and steps
    assert f(steps=A) == gc.GC_ERR_INVALID_ARG
    assert f(cols=0) == gc.GC_ERR_LAYOUT
    assert f(rows=0, x=None, y=None) == gc.GC_OK


def test_rmsnorm_backward_refusals(gc):
    size = C.c_size_t(0)
    assert gc.lib().gc_rmsnorm_backward_workspace_size(100, 64, C.byref(size)) == gc.GC_OK
    need = size.value
    assert need >= 4 * 64

    def f(dy=A, lddy=64, dh=None, lddh=0, dt=1, codes=A, steps=A, rstd=A, w=A, wt=1, rows=100, cols=64, dx=A, lddx=64,
          dw=A, flags=0, ws=A, n=need):
        return gc.lib().gc_rmsnorm_backward(dy, lddy, dh, lddh, dt, codes, steps, rstd, w, wt, rows, cols, dx, lddx, dw,
                                            flags, ws, n, None)

    assert f(ws=None) == gc.GC_ERR_WORKSPACE
    assert f(n=need - 1) == gc.GC_ERR_WORKSPACE
    assert f(ws=A + 128) == gc.GC_ERR_WORKSPACE
    assert f(flags=2) == gc.GC_ERR_INVALID_ARG
    assert f(rstd=None) == gc.GC_ERR_INVALID_ARG
    assert f(codes=None) == gc.GC_ERR_INVALID_ARG
    assert f(dx=None) == gc.GC_ERR_INVALID_ARG
    assert f(lddx=63) == gc.GC_ERR_LAYOUT
    assert f(dh=A, lddh=0) == gc.GC_ERR_LAYOUT
    assert f(dw=A + 1) == gc.GC_ERR_ALIGNMENT


def test_gated_refusals(gc):
    def f(kind=0, g=A, ldg=64, u=A, ldu=64, dt=1, rows=4, cols=64, o=A, ldo=64, gcod=None, gs=None, uc=None, us=None):
        return gc.lib().gc_gated_act(kind, g, ldg, u, ldu, dt, rows, cols, o, ldo, gcod, gs, uc, us, None)

    assert f(kind=2) == gc.GC_ERR_INVALID_ARG
    assert f(u=None) == gc.GC_ERR_INVALID_ARG
    assert f(ldo=60) == gc.GC_ERR_LAYOUT
    assert f(gcod=A, gs=A) == gc.GC_ERR_INVALID_ARG     # both checkpoints or none
    assert f(gcod=A, gs=A, uc=A) == gc.GC_ERR_INVALID_ARG
    assert f(gcod=A, gs=A, uc=A + 4, us=A) == gc.GC_ERR_ALIGNMENT

    def b(kind=0, d=A, ldd=64, dt=1, gcod=A, gs=A, uc=A, us=A, rows=4, cols=64, dg=A, lddg=64, du=A, lddu=64, oc=None,
          os=None):
        return gc.lib().gc_gated_act_backward(kind, d, ldd, dt, gcod, gs, uc, us, rows, cols, dg, lddg, du, lddu, oc,
                                              os, None)

    assert b(kind=-1) == gc.GC_ERR_INVALID_ARG
    assert b(uc=None) == gc.GC_ERR_INVALID_ARG
    assert b(oc=A) == gc.GC_ERR_INVALID_ARG
    assert b(lddu=3) == gc.GC_ERR_LAYOUT
    assert b(dt=9) == gc.GC_ERR_INVALID_ARG
    assert b(rows=0, d=None) == gc.GC_OK


def test_weight_grad_refusals(gc):
    size = C.c_size_t(0)
    for bad in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (8, 1 << 31, 8)):
        assert gc.lib().gc_act_weight_grad_workspace_size(*bad, gc.GC_BF16, C.byref(size)) == gc.GC_ERR_LAYOUT
    assert gc.lib().gc_act_weight_grad_workspace_size(8, 8, 8, 5, C.byref(size)) == gc.GC_ERR_INVALID_ARG
    assert gc.lib().gc_act_weight_grad_workspace_size(8, 8, 8, 0, None) == gc.GC_ERR_INVALID_ARG
    assert gc.lib().gc_act_weight_grad_workspace_size(8192, 64, 64, gc.GC_BF16, C.byref(size)) == gc.GC_OK
    need = size.value

    def f(dy=A, lddy=64, dt=1, rows=8192, n=64, codes=A, steps=A, k=64, cs=None, ct=0, dw=A, lddw=64, flags=0, ws=A,
          nb=need):
        return gc.lib().gc_act_weight_grad(dy, lddy, dt, rows, n, codes, steps, k, cs, ct, dw, lddw, flags, ws, nb, None)

    assert f(dy=None) == gc.GC_ERR_INVALID_ARG
    assert f(lddy=63) == gc.GC_ERR_LAYOUT
    assert f(lddw=63) == gc.GC_ERR_LAYOUT
    assert f(dw=None) == gc.GC_ERR_INVALID_ARG
    assert f(flags=4) == gc.GC_ERR_INVALID_ARG
    assert f(cs=A, ct=3) == gc.GC_ERR_INVALID_ARG
    assert f(codes=A + 8) == gc.GC_ERR_ALIGNMENT
    if need:
        assert f(nb=need - 1) == gc.GC_ERR_WORKSPACE
        assert f(ws=None) == gc.GC_ERR_WORKSPACE


def test_binding_refuses_host_tensors_and_wrong_shapes(gc):
    with pytest.raises(ValueError):
        gc.ActCheckpoint(4, 64, codes=torch.empty(4, 64, dtype=torch.int8), steps=torch.empty(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gc.ActCheckpoint(4, 0)
    with pytest.raises(ValueError):
        gc.gated_act(gc.GC_GATE_SILU, torch.empty(4, 64), torch.empty(4, 64), torch.empty(4, 64))
    with pytest.raises(ValueError):
        gc.rmsnorm(torch.empty(4, 64), None, 1e-5, torch.empty(4, 64))
    with pytest.raises(ValueError):
        gc.act_weight_grad_workspace(8, 8, 8, torch.float64)
