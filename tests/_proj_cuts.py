"""The ways in which the gated projection cuts a call, and sizes that take each."""
import ctypes as C
import math
import os
import random
import subprocess
import tempfile

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
# clusters of 1, 2, ... 8 CTAs of the kernel that a GB300 holds (an SM each)
HELD = (152, 76, 46, 36, 28, 23, 15, 15)
SMS = 152
MODES = ("out", "held", "back")          # the projection without checkpoints, with them, its gradient
LARGE = {"out": [(2048, 4096, 1024), (300, 11136, 3840), (48, 14336, 4096), (64, 5632, 4096), (17, 11136, 3840)],
         "held": [(2048, 4096, 1024), (300, 11136, 3840), (48, 14336, 4096)],
         "back": [(2048, 14336, 4096), (2048, 4096, 1024), (512, 14336, 4096)]}


def library():
    """_proj_plan.cpp, compiled."""
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "libplan.so")
        subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-fPIC", "-shared",
                        os.path.join(HERE, "_proj_plan.cpp"), "-o", out], check=True)
        lib = C.CDLL(out)
    lib.proj_few.argtypes = [C.c_int64] * 3
    lib.proj_stage.argtypes, lib.proj_stage.restype = [C.c_int64, C.c_int, C.c_int, C.c_int], C.c_int64
    return lib


def plans(lib, mode, sizes, held=HELD):
    """pair, apart, bn, parts, tiles_m, tiles_n, splits, span of each of `sizes` (rows, n, k)."""
    calls = np.array([(r, k, n, 1, 0) if mode == "back" else (r, n, k, 0, int(mode == "out")) for r, n, k in sizes], dtype=np.int64)
    cuts = np.zeros((len(sizes), 8), dtype=np.int64)
    lib.proj_plans(calls.ctypes.data_as(C.c_void_p), C.c_int64(len(sizes)), (C.c_int * 9)(0, *held), cuts.ctypes.data_as(C.c_void_p))
    return cuts.tolist()


def kind(lib, mode, size, plan):
    """What of a cut decides which code runs: the kernel, the tile, how the sum is split, whether
    a CTA has several tiles, whether memory's share counted."""
    rows, n, k = size
    if mode == "out" and lib.proj_few(rows, n, k):
        return ("few", min(rows, 3))
    pair, apart, bn, parts, tm, tn, splits, _ = plan
    cols, summed = (k, n) if mode == "back" else (n, k)
    memory = (4 * cols + (4 if mode == "back" else 2) * rows) * summed > 64e6
    return (pair, bn, parts, "apart" if apart else splits, tm * tn * splits > (SMS // 2 if pair else SMS), memory)


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draws(seed, count):
    """Sizes over the range of real calls; widths of any number, or of multiples of 8 or 128."""
    rng, out = random.Random(seed), []
    while len(out) < count:
        rows, n, k = _log_int(rng, 1, 16384), _log_int(rng, 16, 14336), _log_int(rng, 16, 8192)
        m, q = rng.choice((1, 8, 128)), rng.choice((1, 8, 128))
        n, k = -(-n // m) * m, -(-k // q) * q
        if rows * n * k <= 8192 * 14336 * 4096:
            out.append((rows, n, k))
    return out


def kinds(lib, mode, sizes):
    found = {}
    for size, plan in zip(sizes, plans(lib, mode, sizes)):
        found.setdefault(kind(lib, mode, size, plan), []).append(size)
    return found


def cases(lib, mode):
    """{kind: the size of least work that takes it, and one of middling work}"""
    out = {}
    for what, sizes in kinds(lib, mode, draws(59, 40000)).items():
        sizes = sorted(sizes, key=lambda s: s[0] * s[1] * s[2])
        middle = [s for s in sizes if s[0] * s[1] * s[2] <= 10 ** 10] or sizes[:1]
        out[what] = sorted({sizes[0], middle[len(middle) * 3 // 4]})
    for size, plan in zip(LARGE[mode], plans(lib, mode, LARGE[mode])):
        out.setdefault(kind(lib, mode, size, plan), []).append(size)
    return out
