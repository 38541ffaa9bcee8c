"""Gated projection and global gradient norm: arguments refused on the host
before anything is enqueued (CPU only)."""
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


def _size(gc, f, *args):
    size = C.c_size_t(0)
    assert f(*args, C.byref(size)) == gc.GC_OK
    return size.value


def test_workspace_sizes(gc):
    L = gc.lib()
    out = C.c_size_t(0)
    for f in (L.gc_gated_proj_workspace_size, L.gc_gated_proj_backward_workspace_size):
        for bad in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (8, 1 << 31, 8), ((1 << 31) - 1, 1 << 30, 8)):
            assert f(*bad, 0, C.byref(out)) == gc.GC_ERR_LAYOUT
        assert f(8, 8, 8, 4, C.byref(out)) == gc.GC_ERR_INVALID_ARG
        assert f(8, 8, 8, 0, None) == gc.GC_ERR_INVALID_ARG
        for n, k in ((100, 70), (4096, 1024), (14336, 4096), (1, 1)):
            for copied in range(4):
                last = 0
                for rows in (0, 1, 5, 127, 128, 129, 1000, 1031, 2048, 9999, 16384):
                    now = _size(gc, f, rows, n, k, copied)
                    assert now >= last and now >= 256                    # does for fewer rows, too
                    assert now >= 2 * 2 * n * k * (copied >> 1) + (2 * rows * k if copied & 1 and "backward" not in f.__name__ else 0)
                    last = now


def test_gated_proj_refusals(gc):
    need = _size(gc, gc.lib().gc_gated_proj_workspace_size, 4, 40, 64, 0)

    def f(kind=0, x=A, ldx=64, wg=A, ldwg=64, wu=A, ldwu=64, dt=1, rows=4, n=40, k=64, o=A, ldo=40, gcod=None, gs=None,
          uc=None, us=None, ws=A, nb=need):
        return gc.lib().gc_gated_proj(kind, x, ldx, wg, ldwg, wu, ldwu, dt, rows, n, k, o, ldo, gcod, gs, uc, us, ws, nb, None)

    assert f(kind=2) == f(kind=-1) == gc.GC_ERR_INVALID_ARG
    assert f(dt=0) == f(dt=3) == gc.GC_ERR_INVALID_ARG                  # 16-bit types only
    assert f(rows=-1) == f(n=0) == f(k=0) == gc.GC_ERR_LAYOUT
    assert f(x=None) == f(wg=None) == f(wu=None) == f(o=None) == gc.GC_ERR_INVALID_ARG
    assert f(ldx=63) == f(ldwg=63) == f(ldwu=63) == f(ldo=39) == gc.GC_ERR_LAYOUT
    assert f(x=A + 1) == f(o=A + 1) == gc.GC_ERR_ALIGNMENT
    assert f(gcod=A, gs=A) == f(gcod=A) == f(us=A) == gc.GC_ERR_INVALID_ARG
    assert f(gcod=A + 4, gs=A, uc=A, us=A) == gc.GC_ERR_ALIGNMENT
    assert f(ws=None) == f(nb=need - 1) == f(ws=A + 128) == gc.GC_ERR_WORKSPACE
    # rows off 16-byte boundaries need room for copies
    assert f(x=A + 2) == f(ldx=65) == f(wg=A + 8) == f(ldwu=68) == gc.GC_ERR_WORKSPACE


def test_gated_proj_backward_refusals(gc):
    need = _size(gc, gc.lib().gc_gated_proj_backward_workspace_size, 4, 40, 64, 0)

    def f(kind=0, d=A, ldd=40, dt=1, gcod=A, gs=A, uc=A, us=A, wg=A, ldwg=64, wu=A, ldwu=64, rows=4, n=40, k=64, dg=A,
          lddg=40, du=A, lddu=40, dx=A, lddx=64, oc=None, os=None, ws=A, nb=need):
        return gc.lib().gc_gated_proj_backward(kind, d, ldd, dt, gcod, gs, uc, us, wg, ldwg, wu, ldwu, rows, n, k, dg, lddg,
                                               du, lddu, dx, lddx, oc, os, ws, nb, None)

    assert f(kind=2) == f(dt=0) == f(dt=7) == gc.GC_ERR_INVALID_ARG
    assert f(rows=-1) == f(n=0) == f(k=0) == gc.GC_ERR_LAYOUT
    for missing in ("d", "gcod", "gs", "uc", "us", "wg", "wu", "dg", "du", "dx"):
        assert f(**{missing: None}) == gc.GC_ERR_INVALID_ARG, missing
    for ld in ("ldd", "lddg", "lddu"):
        assert f(**{ld: 39}) == gc.GC_ERR_LAYOUT, ld
    for ld in ("ldwg", "ldwu", "lddx"):
        assert f(**{ld: 63}) == gc.GC_ERR_LAYOUT, ld
    assert f(oc=A) == f(os=A) == gc.GC_ERR_INVALID_ARG
    assert f(dx=A + 1) == f(uc=A + 8) == gc.GC_ERR_ALIGNMENT
    assert f(ws=None) == f(nb=need - 1) == f(ws=A + 16) == gc.GC_ERR_WORKSPACE
    assert f(dg=A + 2) == f(lddu=41) == f(wu=A + 2) == gc.GC_ERR_WORKSPACE


def _list(gc, *tensors):
    return (gc.gc_tensor * max(len(tensors), 1))(*[gc.gc_tensor(*t) for t in tensors])


def test_grad_norm_refusals(gc):
    need = _size(gc, gc.lib().gc_grad_norm_workspace_size, 2)
    out = C.c_size_t(0)
    assert gc.lib().gc_grad_norm_workspace_size(-1, C.byref(out)) == gc.GC_ERR_INVALID_ARG
    assert gc.lib().gc_grad_norm_workspace_size(1, None) == gc.GC_ERR_INVALID_ARG
    sizes = [_size(gc, gc.lib().gc_grad_norm_workspace_size, c) for c in (0, 1, 1024, 1025, 5000)]
    assert sizes == sorted(sizes) and sizes[0] > 0

    def f(*tensors, count=None, norm=A, ws=A, nb=need):
        return gc.lib().gc_grad_norm(_list(gc, *tensors), len(tensors) if count is None else count, norm, ws, nb, None)

    good = (A, 5, 0)
    assert f(good, count=-1) == gc.GC_ERR_INVALID_ARG
    assert gc.lib().gc_grad_norm(None, 1, A, A, need, None) == gc.GC_ERR_INVALID_ARG
    assert f((A, 5, 3)) == f((A, 5, -1)) == f((None, 5, 0)) == gc.GC_ERR_INVALID_ARG
    assert f((A, -1, 0)) == f(good, (A, (1 << 42) + 1, 0)) == gc.GC_ERR_LAYOUT
    assert f((A, 1 << 42, 1), (A, 1, 1)) == gc.GC_ERR_LAYOUT
    assert f((A + 2, 5, 0)) == f((A + 1, 5, 1)) == f(good, norm=A + 2) == gc.GC_ERR_ALIGNMENT
    assert f(good, norm=None) == gc.GC_ERR_INVALID_ARG
    assert f(good, ws=None) == f(good, nb=need - 1) == f(good, ws=A + 8) == gc.GC_ERR_WORKSPACE


def test_grad_clip_refusals(gc):
    N = 0x900000

    def f(ins, outs, norm=N, most=1.0, count=None):
        return gc.lib().gc_grad_clip(_list(gc, *ins), _list(gc, *outs), len(ins) if count is None else count, norm, most, None)

    one = [(A, 100, 0)]
    assert f(one, one, most=-1.0) == f(one, one, most=float("nan")) == f(one, one, norm=None) == gc.GC_ERR_INVALID_ARG
    assert f(one, one, norm=N + 1) == gc.GC_ERR_ALIGNMENT
    assert f(one, [(A, 99, 0)]) == gc.GC_ERR_LAYOUT
    assert f(one, [(A, 100, 5)]) == f(one, [(None, 100, 0)]) == gc.GC_ERR_INVALID_ARG
    # written twice, or while another one is read
    two = [(A, 100, 0), (A + 400, 100, 0)]
    assert f(two, [(0x20000, 100, 0), (0x20000, 100, 0)]) == gc.GC_ERR_INVALID_ARG
    assert f(two, [(0x20000, 100, 0), (0x20000 + 396, 100, 0)]) == gc.GC_ERR_INVALID_ARG
    assert f(two, [(0x20000 + 396, 100, 0), (0x20000, 100, 0)]) == gc.GC_ERR_INVALID_ARG
    assert f([two[0], two[0]], [two[0], two[0]]) == gc.GC_ERR_INVALID_ARG     # the same one twice, in place
    assert f(two, two[::-1]) == gc.GC_ERR_INVALID_ARG                        # one written over the other
    assert f(one, [(A, 100, 1)]) == gc.GC_ERR_INVALID_ARG                    # its own memory in another type
    assert f(one, [(A + 4, 100, 0)]) == gc.GC_ERR_INVALID_ARG
    assert f(two, [(0x20000, 100, 0), (A + 796, 100, 0)]) == gc.GC_ERR_INVALID_ARG
    assert f(one, one, norm=A + 396) == f(one, [(0x20000, 100, 0)], norm=0x20000) == gc.GC_ERR_INVALID_ARG
    assert f([(None, 0, 0)], [(None, 0, 1)]) == gc.GC_OK                      # nothing to do
    assert f([], []) == gc.GC_OK


def test_binding_refusals(gc):
    host = torch.zeros(4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: gc.gated_proj(0, host, host, host, host, ws),
                 lambda: gc.gated_proj_backward(0, host, host, host, host, host, host, host, host, ws),
                 lambda: gc.gated_proj(0, None, host, host, host, ws), lambda: gc.gated_proj(0, host, "x", host, host, ws),
                 lambda: gc.gated_proj_workspace(host[0], host, host), lambda: gc.gated_proj_workspace(host, None, host),
                 lambda: gc.grad_norm([host], torch.zeros(1), ws), lambda: gc.grad_norm(3, torch.zeros(1), ws),
                 lambda: gc.grad_norm([host], None, ws), lambda: gc.grad_norm([None], torch.zeros(1), ws),
                 lambda: gc.grad_clip([host], torch.zeros(1), 1.0), lambda: gc.grad_clip([host], None, 1.0),
                 lambda: gc.grad_clip(host, 1.0, 1.0), lambda: gc.grad_norm(host, torch.zeros(1), ws),
                 lambda: gc.grad_norm((t for t in [host]), torch.zeros(1), ws)):
        with pytest.raises(ValueError):
            call()
    assert gc.grad_norm_workspace([host, host], device="cpu").numel() >= 8
