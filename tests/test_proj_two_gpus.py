"""What the gated projection asks of a GPU once (shared memory for a kernel),
asked on every GPU, and again where it failed, without leaving an error behind:
against a fake of the CUDA runtime, in a process that sees no GPU."""
import os
import subprocess
import sys

import pytest

from test_act_two_gpus import HERE, fake  # noqa: F401

SCRIPT = r"""
import ctypes as C, sys
fake = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)      # before libgc, whose calls it takes
sys.path.insert(0, sys.argv[2])
import gradient_compression_gb300 as gc
L = gc.lib()
A = 0x10000
OK, CUDA = gc.GC_OK, gc.GC_ERR_CUDA


def proj(kind, dt, rows, n, k, held, ld=0):
    size = C.c_size_t(0)
    assert L.gc_gated_proj_workspace_size(rows, n, k, 3, C.byref(size)) == OK
    c = [A] * 4 if held else [None] * 4
    return lambda: L.gc_gated_proj(kind, A, k + ld, A, k + ld, A, k + ld, dt, rows, n, k, A, n, *c, A, size, None)


def back(dt, rows, n, k, ld=0):
    size = C.c_size_t(0)
    assert L.gc_gated_proj_backward_workspace_size(rows, n, k, 3, C.byref(size)) == OK
    return lambda: L.gc_gated_proj_backward(0, A, n, dt, A, A, A, A, A, k + ld, A, k + ld, rows, n, k, A, n + ld, A, n + ld, A, k, None, None,
                                            A, size, None)


calls = [proj(0, 1, 48, 512, 512, False), proj(1, 1, 48, 512, 512, True), proj(0, 2, 500, 512, 64, True), proj(1, 2, 2000, 4096, 1024, False),
         proj(0, 1, 500, 512, 512, True, 3), back(1, 48, 512, 512), back(2, 500, 512, 512), back(1, 4000, 4096, 1024), back(1, 500, 512, 512, 3)]  # a kernel each
one = proj(0, 1, 1, 512, 512, False)                 # asks nothing
assert one() == OK
for f in calls:
    if sys.argv[3] == "two":
        for gpu in (0, 1, 0):
            fake.fake_device(gpu)
            assert f() == OK, (calls.index(f), gpu)
    else:
        fake.fake_failing(1)
        assert f() == CUDA, calls.index(f)
        fake.fake_failing(0)
        assert one() == OK and f() == OK, calls.index(f)   # this call's error is not the next one's
print("done")
"""


@pytest.mark.parametrize("what", ["two", "again"])
def test_asked_on_every_gpu(fake, what):  # noqa: F811
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    p = subprocess.run([sys.executable, "-c", SCRIPT, fake, os.path.dirname(HERE), what], env=env, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0 and "done" in p.stdout, p.stderr[-2000:]
