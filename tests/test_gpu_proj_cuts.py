"""The gated projection and its gradient in every way in which calls are cut.

Inputs are small integers, so that every sum is exact in fp32 in whatever
order, and what is left is what the activation does to it (within 2^-16 of its
value) and the roundings of the results.  Below 2^-126 fp32 has steps of 2^-149: the
sigmoid of G < -87, its product with G and that with U are half of one off at
most, 2^-150 (|G U| + |U| + 1) in all.  The gradient's G is 64, where silu is
64 and its derivative 1 in fp32: dgate = dout U and dup = 64 dout are exact, and
so is dx before its rounding: its terms' absolute sum stays below 2^24.
"""
import pytest
import torch

import _proj_cuts as cuts

pytestmark = pytest.mark.gpu

TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


@pytest.fixture(scope="module")
def cases():
    lib = cuts.library()
    return {mode: cuts.cases(lib, mode) for mode in cuts.MODES}


def integers(gen, rows, cols, most):
    return torch.randint(-most, most + 1, (rows, cols), generator=gen, device="cuda", dtype=torch.int8)


def double_sum(a, b):
    return (a.double() @ b.double().T)


def check_out(gc, size, dt, held):
    rows, n, k = size
    gen = torch.Generator(device="cuda").manual_seed(rows * 31 + n * 7 + k)
    x, w = integers(gen, rows, k, 1), integers(gen, 2 * n, k, 1)
    xd, wd = x.to(dt), w.to(dt)
    out = torch.full((rows, n), 77.0, dtype=dt, device="cuda")
    ws = gc.gated_proj_workspace(xd, wd[:n], wd[n:])
    cks = [gc.ActCheckpoint(rows, n) for _ in range(2)] if held else []
    gc.gated_proj(gc.GC_GATE_SILU, xd, wd[:n], wd[n:], out, ws, *cks)
    assert gc.get_device_status(ws).error_bits == 0
    g, u = double_sum(x, w[:n]), double_sum(x, w[n:])
    for ck, full in zip(cks, (g, u)):
        ref = gc.ActCheckpoint(rows, n)
        gc.act_compress(full.float(), ref)
        assert torch.equal(ck.codes, ref.codes) and torch.equal(ck.steps, ref.steps), size
    want = g * torch.sigmoid(g) * u
    error = 2.0 ** -16 * want.abs() + 2.0 ** -150 * ((g * u).abs() + u.abs() + 1)
    top = torch.finfo(dt).max
    assert float(want.abs().max()) < top
    off = (out.double() - want).abs() - (error + (want.abs() + error) * (torch.finfo(dt).eps / 2) + TINY[dt] / 2)
    assert float(off.max()) <= 0.0, (size, float(off.max()))


def check_back(gc, size, dt):
    rows, n, k = size
    gen = torch.Generator(device="cuda").manual_seed(rows * 31 + n * 7 + k)
    d, u, w = integers(gen, rows, n, 1), integers(gen, rows, n, 2), integers(gen, 2 * n, k, 1)
    cg, cu = gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)
    gc.act_compress(torch.full((rows, n), 64.0, dtype=dt, device="cuda"), cg)
    gc.act_compress(u.to(dt), cu)
    dout, wd = d.to(dt), w.to(dt)
    dgate, dup, dx = (torch.full((rows, c), 77.0, dtype=dt, device="cuda") for c in (n, n, k))
    ws = gc.gated_proj_backward_workspace(dgate, dup, wd[:n], wd[n:])
    gc.gated_proj_backward(gc.GC_GATE_SILU, dout, cg, cu, wd[:n], wd[n:], dgate, dup, dx, ws)
    assert gc.get_device_status(ws).error_bits == 0
    assert torch.equal(dgate, (d * u).to(dt)) and torch.equal(dup, 64 * dout), size
    want = double_sum(d * u, w[:n].T) + 64 * double_sum(d, w[n:].T)
    assert float(want.abs().max()) < torch.finfo(dt).max
    assert torch.equal(dx, want.to(dt)), size


OUT = ["few"] + [(pair, bn) for pair in (0, 1) for bn in range(32, 129, 16)]
HELD = [(pair, bn) for pair in (0, 1) for bn in range(32, 129, 32)]
BACK = [(pair, bn) for pair in (0, 1) for bn in range(32, 257, 32)]


def dtype(i, sum_over):
    """Half of them fp16, where six standard deviations of a projection, squared, are in its range."""
    return torch.float16 if i % 2 and 16 * sum_over < torch.finfo(torch.float16).max else torch.bfloat16


def some(cases, mode, which):
    found = [(what, size) for what, sizes in cases[mode].items() for size in sizes
             if (what[0] if which == "few" else what[:2]) == which]
    assert found
    return sorted(found, key=str)


def name(which):
    return which if which == "few" else "%s%d" % ("pair" if which[0] else "single", which[1])


@pytest.mark.parametrize("which", OUT, ids=name)
def test_projection(gc, cases, which):
    for i, (_, size) in enumerate(some(cases, "out", which)):
        check_out(gc, size, dtype(i, size[2]), False)


@pytest.mark.parametrize("which", HELD, ids=name)
def test_projection_with_checkpoints(gc, cases, which):
    for i, (_, size) in enumerate(some(cases, "held", which)):
        check_out(gc, size, dtype(i, size[2]), True)


@pytest.mark.parametrize("which", BACK, ids=name)
def test_gradient(gc, cases, which):
    for i, (_, size) in enumerate(some(cases, "back", which)):
        check_back(gc, size, dtype(i, 0))
