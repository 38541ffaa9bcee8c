"""What the activation entry points ask of a GPU once (shared memory for a
kernel, how many of its CTAs an SM holds), asked on every GPU, and again where
it failed: against a fake of the CUDA runtime, in a process that sees no GPU."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

SCRIPT = r"""
import ctypes as C, sys
fake = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)      # before libgc, whose calls it takes
sys.path.insert(0, sys.argv[2])
import gradient_compression_gb300 as gc
L = gc.lib()
A = 0x10000
OK, CUDA = gc.GC_OK, gc.GC_ERR_CUDA


def norm(dtype, cols, odd=0):
    return lambda: L.gc_rmsnorm(A + 4 * odd, cols, None, 0, dtype, A, dtype, 1e-5, 100, cols, A, cols, None, 0, None, None, None, None)


def norm_backward(dtype, cols):
    return lambda: L.gc_rmsnorm_backward(A, cols, None, 0, dtype, A, A, A, None, 0, 100, cols, A, cols, None, 0, None, 0, None)


def weight_grad(dtype, n, lddy):
    size = C.c_size_t(0)
    assert L.gc_act_weight_grad_workspace_size(500, n, 600, dtype, C.byref(size)) == OK
    return lambda: L.gc_act_weight_grad(A, lddy, dtype, 500, n, A, A, 600, None, 0, A, 600, 0, A, size, None)


calls = [norm(0, 9000), norm(0, 5000), norm(1, 8192), norm(1, 5000), norm(1, 16384), norm(2, 12296), norm(1, 5001, 1),
         norm_backward(0, 9000), norm_backward(1, 8192), norm_backward(2, 5000), norm_backward(1, 9001),
         weight_grad(0, 304, 304), weight_grad(1, 304, 304), weight_grad(1, 304, 305), weight_grad(2, 304, 304)]
if sys.argv[3] == "two":
    for f in calls:
        for gpu in (0, 1, 0):
            fake.fake_device(gpu)
            assert f() == OK, (calls.index(f), gpu)
elif sys.argv[3] == "again":
    for f in calls:
        fake.fake_failing(1)
        assert f() == CUDA, calls.index(f)
        fake.fake_failing(0)
        assert f() == OK, calls.index(f)
else:
    grids = []
    for gpu in (0, 1, 0):
        fake.fake_device(gpu)
        assert L.gc_gated_act(0, A, 4096, A, 4096, 1, 3000, 4096, A, 4096, None, None, None, None, None) == OK
        grids.append(fake.fake_grid_y())
    # 2 and 5 CTAs on each of 152 SMs, two across: slabs of 20 and of 8 rows
    assert grids == [150, 375, 150], grids
print("done")
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from gradient_compression_gb300 import build
    build.build()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    out = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-fPIC", "-shared", "-I", os.path.join(cuda, "include"),
                    os.path.join(HERE, "_fake_cudart.cpp"), "-o", out], check=True)
    return out


@pytest.mark.parametrize("what", ["two", "again", "held"])
def test_asked_on_every_gpu(fake, what):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    p = subprocess.run([sys.executable, "-c", SCRIPT, fake, os.path.dirname(HERE), what], env=env, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0 and "done" in p.stdout, p.stderr[-2000:]
