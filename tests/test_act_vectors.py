"""Vectors off their elements' boundaries are refused before anything is
enqueued, as matrices are (CPU only; A stands for an aligned device address)."""
import ctypes as C

import pytest

A = 0x10000


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    gcmod.lib()
    return gcmod


OFF = [(0, 1), (0, 2), (0, 3), (1, 1), (2, 1)]           # type, bytes off


@pytest.mark.parametrize("wtype, off", OFF)
def test_weight_of_the_norm(gc, wtype, off):
    for cols in (64, 20000):
        assert gc.lib().gc_rmsnorm(A, cols, None, 0, 1, A + off, wtype, 1e-5, 4, cols, A, cols, None, 0, None, None, None,
                                   None) == gc.GC_ERR_ALIGNMENT
        assert gc.lib().gc_rmsnorm_backward(A, cols, None, 0, 1, A, A, A, A + off, wtype, 4, cols, A, cols, None, 0, None, 0,
                                            None) == gc.GC_ERR_ALIGNMENT


@pytest.mark.parametrize("off", [1, 2, 3])
def test_rstd(gc, off):
    assert gc.lib().gc_rmsnorm(A, 64, None, 0, 1, None, 0, 1e-5, 4, 64, A, 64, None, 0, A + off, None, None,
                               None) == gc.GC_ERR_ALIGNMENT
    assert gc.lib().gc_rmsnorm_backward(A, 64, None, 0, 1, A, A, A + off, None, 0, 4, 64, A, 64, None, 0, None, 0,
                                        None) == gc.GC_ERR_ALIGNMENT


@pytest.mark.parametrize("wtype, off", OFF)
def test_column_scale(gc, wtype, off):
    size = C.c_size_t(0)
    assert gc.lib().gc_act_weight_grad_workspace_size(40, 64, 64, 1, C.byref(size)) == gc.GC_OK
    assert gc.lib().gc_act_weight_grad(A, 64, 1, 40, 64, A, A, 64, A + off, wtype, A, 64, 0, A, size.value,
                                       None) == gc.GC_ERR_ALIGNMENT
    # without rows the result is still scaled
    assert gc.lib().gc_act_weight_grad(None, 64, 1, 0, 64, None, None, 64, A + off, wtype, A, 64, 0, A, size.value,
                                       None) == gc.GC_ERR_ALIGNMENT
