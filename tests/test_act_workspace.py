"""Workspaces of the activation operators: what was set aside for a batch holds
every smaller one (the last of an epoch, say).  CPU only."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    gcmod.lib()
    return gcmod


def size(f, *args):
    out = C.c_size_t(0)
    assert f(*args, C.byref(out)) == 0
    return out.value


ROWS = sorted(set(range(0, 17000, 13)) | set(range(64, 17000, 64)) | set(range(65, 17000, 64)) | {1, 2, 3, 40000, 65536, 10 ** 6})


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("n, k", [(1, 1), (64, 64), (333, 1001), (512, 512), (768, 768), (1024, 1024), (2048, 1111),
                                  (1500, 2600), (4096, 4096), (136, 14336)])
def test_weight_grad_workspace_never_falls_as_rows_grow(gc, n, k, dtype):
    f = gc.lib().gc_act_weight_grad_workspace_size
    sizes = [size(f, r, n, k, dtype) for r in ROWS]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    # all but dy's terms and the diagnostic words are partial sums, of at most one
    # tile for each of 152 SMs
    terms = {0: 3, 1: 1, 2: 2}[dtype] * 2 * ((n + 7) // 8 * 8)
    assert all(s <= 512 + r * terms + 152 * 256 * 256 * 4 for r, s in zip(ROWS, sizes))


@pytest.mark.parametrize("cols", [1, 100, 512, 1024, 5000, 8192, 16384, 20000])
def test_norm_workspace_never_falls_as_rows_grow(gc, cols):
    f = gc.lib().gc_rmsnorm_backward_workspace_size
    sizes = [size(f, r, cols) for r in ROWS]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
