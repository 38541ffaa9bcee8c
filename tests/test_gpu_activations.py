"""Activation checkpoints, RMS norm, gated activation and weight gradient
against plain 64-bit forms.

Tolerances.  u = 2^-24 (fp32's unit roundoff).  An output is the rounding to
its type of a value computed in fp32, so it lies between the roundings of the
64-bit value's lower and upper bound; no constant of the type is needed.
Codes and steps of a matrix given as it is are exact: |x| / step is exact and
rounded once.  Values computed in fp32 before they are held carry a relative
error of at most about (8 + log2 cols) u from a tree or fused sum; it is taken
as 2^-18 of the terms' absolute sum throughout, far above that and far below
a code's half step (2^-8).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = 2.0 ** -18
SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 100), (7, 257), (4, 1000), (3, 1024), (2, 4097), (33, 136),
          (1, 4096), (2, 14336), (2, 20000)]


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


# -------------------------------------------------------------------- 64-bit forms

def held(x):
    """(codes, step bytes, values) of float64 x[rows, cols], from the definition."""
    rows, cols = x.shape
    ldc = (cols + 31) // 32 * 32
    p = np.zeros((rows, ldc))
    p[:, :cols] = x
    g = p.reshape(rows, -1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(g).max(2)
        bad = ~np.isfinite(top)
        t = np.where(bad, 0.0, top)
        b = np.frexp(t)[1] - 7                                   # t / 2^b in [64, 128)
        b = b + (np.rint(t / np.exp2(b.astype(float))) > 127)
        b = np.clip(b + 127, 1, 248)
        b = np.where(t == 0, 1, b)
        step = np.exp2(b - 127.0)[..., None]
        codes = np.where(bad[..., None], 0, np.clip(np.rint(np.where(bad[..., None], 0, g) / step), -127, 127))
    values = np.where(bad[..., None], np.nan, codes * step)
    return (codes.reshape(rows, ldc).astype(np.int8), np.where(bad, 255, b).astype(np.uint8),
            values.reshape(rows, ldc)[:, :cols])


def read(ck):
    step = np.exp2(ck.steps.cpu().numpy().astype(np.float64) - 127).repeat(32, 1)
    return (ck.codes.cpu().numpy().astype(np.float64) * step)[:, :ck.cols]


def act64(kind, g):
    """(act, act') in 64 bits: SiLU or the tanh form of GELU."""
    with np.errstate(over="ignore"):
        if kind == 0:
            s = 1 / (1 + np.exp(-g))
            return g * s, s + g * s * (1 - s)
        # (1 + tanh z) / 2 = 1 / (1 + exp(-2z)): no cancellation far out on the left
        c = 2 * math.sqrt(2 / math.pi)
        p = c * (g + 0.044715 * g ** 3)
        s = 1 / (1 + np.exp(-p))
        return g * s, s + g * s / (1 + np.exp(p)) * c * (1 + 3 * 0.044715 * g * g)


def f64(t):
    return t.double().cpu().numpy()


def near(got, want, dtype, terms, what):
    """got is the rounding to its type of a number within 2^-18 of the terms'
    sizes of want."""
    got, room = f64(got), REL * terms + 1e-38
    low = f64(torch.from_numpy(np.asarray(want - room)).to(DT[dtype]))
    high = f64(torch.from_numpy(np.asarray(want + room)).to(DT[dtype]))
    bad = ~((low <= got) & (got <= high))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], np.asarray(want)[bad][:4])


def holds(ck, want, what):
    """A checkpoint of fp32-computed values: the 64-bit values within half of
    the group's step (and the fp32 error), pad codes 0, the step the 64-bit
    one except next to a boundary."""
    codes, steps, _ = held(want)
    got = ck.steps.cpu().numpy()
    up = held(want * (1 + REL))[1]
    down = held(want * (1 - REL))[1]
    assert ((got == steps) | (got == up) | (got == down)).all(), what
    step = np.exp2(got.astype(np.float64) - 127).repeat(32, 1)[:, :ck.cols]
    assert (np.abs(read(ck) - want) <= 0.5 * step + REL * np.abs(want)).all(), what
    assert (ck.codes.cpu().numpy()[:, ck.cols:] == 0).all(), what


def matrix(rows, cols, dtype, seed, layout="plain", size=1.0, channels=True):
    """A matrix of unequal channels, in one of several memory layouts."""
    g = torch.Generator().manual_seed(seed)
    x = size * torch.randn(rows, cols, generator=g)
    if channels:
        x *= torch.exp(0.7 * torch.randn(cols, generator=g))
    return place(x.to(DT[dtype]), layout)


def place(x, layout):
    rows, cols = x.shape
    if layout == "plain":
        return x.cuda()
    pad, off = {"wide": (24, 8), "odd": (3, 1)}[layout]          # row stride cols + pad, first column at off
    buf = torch.full((rows, cols + pad), 77.0, dtype=x.dtype).cuda()
    buf[:, off:off + cols] = x.cuda()
    return buf[:, off:off + cols]


def untouched(view):
    """The columns around a placed matrix still hold what they held."""
    buf = view._base
    if buf is None or buf.shape == view.shape:
        return True
    off = view.storage_offset()
    keep = torch.ones(buf.shape[1], dtype=torch.bool)
    keep[off:off + view.shape[1]] = False
    return bool((buf[:, keep.cuda()] == 77.0).all())


LAYOUTS = ["plain", "wide", "odd"]


# ------------------------------------------------------------------------ checkpoints

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
def test_compress_and_decompress_are_exact(gc, shape, dtype, layout):
    x = matrix(*shape, dtype, 1, layout)
    ck = gc.ActCheckpoint(*shape)
    gc.act_compress(x, ck)
    codes, steps, values = held(f64(x))
    assert np.array_equal(ck.steps.cpu().numpy(), steps)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    for out_type in DT:
        out = place(torch.zeros(*shape, dtype=DT[out_type]), layout)
        gc.act_decompress(ck, out)
        want = torch.from_numpy(values).to(DT[out_type])          # one rounding (fp16's subnormals)
        assert torch.equal(out.cpu(), want)
        assert untouched(out)


def test_special_groups(gc):
    rows = [torch.zeros(64)]
    for first in (float("nan"), float("inf"), -float("inf"), 3.4028234663852886e38, -3.3e38, 1e-45, 1.17e-38, 127.5,
                  -127.5, 127.49999, 127.0, 128.0, 255.0, 2.0 ** -120, 2.0 ** 126):
        r = torch.linspace(-3, 3, 64)
        r[:32] *= abs(first) / 4 if math.isfinite(first) else 1.0
        r[5] = first
        rows.append(r)
    ties = torch.arange(64, dtype=torch.float32) - 31.5                        # halves: ties go to the even code
    ties[0] = ties[32] = 100.0
    rows += [ties, -ties]
    x = torch.stack(rows).cuda()
    ck = gc.ActCheckpoint(*x.shape)
    gc.act_compress(x, ck)
    codes, steps, values = held(f64(x))
    assert np.array_equal(ck.steps.cpu().numpy(), steps)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    out = torch.empty_like(x)
    gc.act_decompress(ck, out)
    assert np.array_equal(f64(out), values, equal_nan=True)
    assert np.isnan(values[1:4, :32]).all() and np.isfinite(values[1:4, 32:]).all()


# ------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
def test_rmsnorm(gc, shape, dtype, layout):
    rows, cols = shape
    x, r = matrix(rows, cols, dtype, 2, layout), matrix(rows, cols, dtype, 3, layout)
    for residual, wtype, keep in ((r, dtype, True), (None, "f32", True), (r, "f32", False), (None, None, False)):
        w = None if wtype is None else (1 + 0.2 * torch.randn(cols)).to(DT[wtype]).cuda()
        y, h = place(torch.zeros(rows, cols, dtype=DT[dtype]), layout), place(torch.zeros(rows, cols, dtype=DT[dtype]), layout)
        rstd = torch.zeros(rows, device="cuda")
        ck = gc.ActCheckpoint(rows, cols) if keep else None
        gc.rmsnorm(x, w, 1e-5, y, residual=residual, h=h, rstd=rstd, ckpt=ck)
        hw = f64(x) + (0 if residual is None else f64(residual))
        rs = 1 / np.sqrt((hw * hw).mean(1) + 1e-5)
        size = np.abs(f64(x)) + (0 if residual is None else np.abs(f64(residual)))
        xh, xsize = hw * rs[:, None], size * rs[:, None]
        ww = 1.0 if w is None else f64(w)
        near(h, hw, dtype, size, "h")
        near(rstd, rs, "f32", rs, "rstd")
        near(y, xh * ww, dtype, xsize * np.abs(ww), "y")
        if keep:
            holds(ck, xh, "checkpoint")
        assert untouched(y) and untouched(h)
        y2 = torch.empty_like(y)                                   # without the other outputs: the same bits
        gc.rmsnorm(x, w, 1e-5, y2, residual=residual)
        assert torch.equal(y2, y)


def test_rmsnorm_in_place(gc):
    x, r = matrix(37, 1000, "bf16", 4), matrix(37, 1000, "bf16", 5)
    w = torch.randn(1000).cuda()
    y, h = torch.empty_like(x), torch.empty_like(x)
    gc.rmsnorm(x, w, 1e-6, y, residual=r, h=h)
    x2, r2 = x.clone(), r.clone()
    gc.rmsnorm(x2, w, 1e-6, x2, residual=r2, h=r2)                 # y over x, h over the residual
    assert torch.equal(x2, y) and torch.equal(r2, h)


def test_rmsnorm_rows_of_zeros_and_nan(gc):
    x = matrix(4, 96, "bf16", 6)
    x[1] = 0
    x[2, 40] = float("nan")
    y, ck = torch.empty_like(x), gc.ActCheckpoint(4, 96)
    gc.rmsnorm(x, None, 1e-5, y, ckpt=ck)
    assert torch.equal(y[1], torch.zeros_like(y[1])) and bool(torch.isnan(y[2]).all())
    assert (ck.codes[1] == 0).all() and (ck.steps[1] == 1).all() and (ck.steps[2] == 255).all()
    assert bool(torch.isfinite(y[[0, 3]]).all())


def norm_backward64(dy, q, rstd, w, dh):
    gw = dy * w
    c = (gw * q).mean(1, keepdims=True)
    dx = rstd[:, None] * (gw - q * c) + dh
    size = rstd[:, None] * (np.abs(gw) + np.abs(q) * np.abs(gw * q).mean(1, keepdims=True)) + np.abs(dh)
    return dx, size, (dy * q).sum(0), np.abs(dy * q).sum(0)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES + [(1000, 64), (300, 777)])
def test_rmsnorm_backward(gc, shape, dtype, layout):
    rows, cols = shape
    ck = gc.ActCheckpoint(rows, cols)
    gc.act_compress(matrix(rows, cols, "f32", 7), ck)
    rstd = (0.5 + torch.rand(rows)).cuda()
    dy, dh = matrix(rows, cols, dtype, 8, layout, 0.1), matrix(rows, cols, dtype, 9, layout, 0.1)
    dy[0] = 0                                                      # a masked token
    w = (1 + 0.2 * torch.randn(cols)).to(DT[dtype]).cuda()
    ws = gc.rmsnorm_backward_workspace(rows, cols)
    for weight, up in ((w, dh), (None, None)):
        dx = place(torch.zeros(rows, cols, dtype=DT[dtype]), layout)
        dw = torch.full((cols,), 7.0, device="cuda")
        gc.rmsnorm_backward(dy, ck, rstd, weight, dx, dw, ws, dh=up)
        want, size, wdw, sdw = norm_backward64(f64(dy), read(ck), f64(rstd), 1.0 if weight is None else f64(weight),
                                               0.0 if up is None else f64(up))
        near(dx, want, dtype, size, "dx")
        near(dw, wdw, "f32", sdw, "dw")
        assert untouched(dx)
        again, dw2 = torch.empty_like(dx), torch.full((cols,), 7.0, device="cuda")
        gc.rmsnorm_backward(dy, ck, rstd, weight, again, dw2, ws, dh=up, accumulate=True)
        assert torch.equal(again, dx)
        assert torch.equal(dw2, dw + 7.0)                          # the same sum, then one addition
        only = torch.empty_like(dx)
        gc.rmsnorm_backward(dy, ck, rstd, weight, only, None, None, dh=up)
        assert torch.equal(only, dx)
    over = dy.clone()
    gc.rmsnorm_backward(over, ck, rstd, None, over, None, None)    # dx over dy
    assert torch.equal(over, dx)


def test_rmsnorm_gradient_against_differences(gc):
    """Central differences of the 64-bit norm; the checkpoint's values are
    within half a step of the normalised rows, so dx and dw are within the
    formula's change under such a perturbation (plus the differences' own
    error, below 1e-7 for a step of 1e-5 in these sizes)."""
    rows, cols = 3, 70
    x = matrix(rows, cols, "f32", 10)
    w = (1 + 0.2 * torch.randn(cols)).cuda()
    dy = matrix(rows, cols, "f32", 11)
    ck, rstd, y = gc.ActCheckpoint(rows, cols), torch.empty(rows, device="cuda"), torch.empty_like(x)
    gc.rmsnorm(x, w, 1e-5, y, rstd=rstd, ckpt=ck)
    dx, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
    gc.rmsnorm_backward(dy, ck, rstd, w, dx, dw, gc.rmsnorm_backward_workspace(rows, cols))

    def loss(xx, ww):
        rs = 1 / np.sqrt((xx * xx).mean(1, keepdims=True) + 1e-5)
        return (f64(dy) * xx * rs * ww).sum()

    x0, w0, e = f64(x), f64(w), 1e-5
    half = 0.5 * np.exp2(ck.steps.cpu().numpy().astype(np.float64) - 127).repeat(32, 1)[:, :cols] * (1 + 1e-4)
    gw, q, rs = f64(dy) * w0, np.abs(read(ck)) + half, f64(rstd)[:, None]
    room = rs * (half * np.abs((gw * read(ck)).mean(1, keepdims=True)) + q * (np.abs(gw) * half).mean(1, keepdims=True))
    for r in range(rows):
        for c in range(cols):
            d = np.zeros_like(x0)
            d[r, c] = e
            diff = (loss(x0 + d, w0) - loss(x0 - d, w0)) / (2 * e)
            assert abs(diff - f64(dx)[r, c]) <= room[r, c] + 1e-6
    for c in range(cols):
        d = np.zeros_like(w0)
        d[c] = e
        diff = (loss(x0, w0 + d) - loss(x0, w0 - d)) / (2 * e)
        assert abs(diff - f64(dw)[c]) <= (np.abs(f64(dy)) * half).sum(0)[c] + 1e-6


# ------------------------------------------------------------------------------ gated

@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
def test_gated(gc, shape, dtype, kind):
    rows, cols = shape
    both = matrix(rows, 2 * cols, dtype, 12)                       # one projection's output: gate, then up
    views = [(both[:, :cols], both[:, cols:], "plain")]
    views += [(matrix(rows, cols, dtype, 13, "odd"), matrix(rows, cols, dtype, 14, "odd"), "odd")]
    for gate, up, layout in views:
        out = place(torch.zeros(rows, cols, dtype=DT[dtype]), layout)
        cg, cu = gc.ActCheckpoint(rows, cols), gc.ActCheckpoint(rows, cols)
        gc.gated_act(kind, gate, up, out, ckpt_gate=cg, ckpt_up=cu)
        g, u = f64(gate), f64(up)
        near(out, act64(kind, g)[0] * u, dtype, np.abs(act64(kind, g)[0] * u), "out")
        for ck, v in ((cg, g), (cu, u)):
            codes, steps, _ = held(v)
            assert np.array_equal(ck.codes.cpu().numpy(), codes) and np.array_equal(ck.steps.cpu().numpy(), steps)
        serve = torch.empty_like(out)
        gc.gated_act(kind, gate, up, serve)
        assert torch.equal(serve, out) and untouched(out)
        dout = matrix(rows, cols, dtype, 15, layout, 0.1)
        dg, du = place(torch.zeros(rows, cols, dtype=DT[dtype]), layout), place(torch.zeros(rows, cols, dtype=DT[dtype]), layout)
        co = gc.ActCheckpoint(rows, cols)
        gc.gated_act_backward(kind, dout, cg, cu, dg, du, ckpt_out=co)
        G, U, d = read(cg), read(cu), f64(dout)
        a, da = act64(kind, G)
        # s + g s (1 - s) p' may cancel: its terms are at most 1 + |g p'(g)| in size where s (1 - s) is not 0
        near(dg, d * U * da, dtype, np.abs(d * U) * (1 + np.abs(da) + np.abs(a)), "dgate")
        near(du, d * a, dtype, np.abs(d * a), "dup")
        holds(co, a * U, "out checkpoint")
        dg2, du2 = torch.empty_like(dg), torch.empty_like(du)
        gc.gated_act_backward(kind, dout, cg, cu, dg2, du2)
        assert torch.equal(dg2, dg) and torch.equal(du2, du) and untouched(dg) and untouched(du)


@pytest.mark.parametrize("kind", [0, 1])
def test_gated_gradient_against_differences(gc, kind):
    """The gradient is taken at the checkpoints' values, so differences of
    the 64-bit activation there give it up to fp32 rounding and the
    differences' own error (below 1e-8 for a step of 1e-5)."""
    g, u, d = matrix(3, 77, "f32", 16), matrix(3, 77, "f32", 17), matrix(3, 77, "f32", 18)
    cg, cu = gc.ActCheckpoint(3, 77), gc.ActCheckpoint(3, 77)
    out, dg, du = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    gc.gated_act(kind, g, u, out, ckpt_gate=cg, ckpt_up=cu)
    gc.gated_act_backward(kind, d, cg, cu, dg, du)
    G, U, e = read(cg), read(cu), 1e-5
    diff_g = f64(d) * U * (act64(kind, G + e)[0] - act64(kind, G - e)[0]) / (2 * e)
    diff_u = f64(d) * act64(kind, G)[0] * ((U + e) - (U - e)) / (2 * e)
    size = np.abs(f64(d)) * (1 + np.abs(G)) * (1 + np.abs(U))
    assert (np.abs(diff_g - f64(dg)) <= (REL + 1e-8) * size).all()
    assert (np.abs(diff_u - f64(du)) <= (REL + 1e-8) * size).all()


@pytest.mark.parametrize("kind", [0, 1])
def test_gated_extremes(gc, kind):
    """Gates so large that the exponential overflows or vanishes, a NaN and an
    infinity: finite where the formula is, and confined to their group."""
    g = torch.tensor([[-1e4, -300.0, -90.0, -30.0, 0.0, -0.0, 30.0, 90.0, 1e4] + [1.0] * 55]).cuda()
    g[0, 40], g[0, 41] = float("nan"), float("inf")
    u = torch.ones_like(g)
    out, dg, du = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    cg, cu = gc.ActCheckpoint(1, 64), gc.ActCheckpoint(1, 64)
    gc.gated_act(kind, g, u, out, ckpt_gate=cg, ckpt_up=cu)
    gc.gated_act_backward(kind, u, cg, cu, dg, du)
    want = act64(kind, f64(g)[:, :32])[0]
    assert (np.abs(f64(out)[:, :32] - want) <= 2.0 ** -18 * np.abs(want) + 1e-30).all()
    assert np.isnan(f64(out)[0, 40]) and f64(out)[0, 41] == np.inf
    assert np.isfinite(f64(dg)[:, :32]).all() and np.isfinite(f64(du)[:, :32]).all()
    assert np.isnan(f64(dg)[:, 32:]).all()
    assert cg.steps[0, 1] == 255 and cu.steps[0, 1] != 255


# ------------------------------------------------------------------------ weight grad

WG = [(1, 1, 1), (1, 64, 64), (2, 17, 33), (15, 128, 256), (64, 256, 256), (65, 257, 255), (130, 300, 1000),
      (257, 8, 4096), (1000, 333, 1001), (512, 1024, 512), (3000, 64, 64), (4096, 136, 72), (8192, 256, 128),
      (100, 2048, 2048)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", WG)
def test_weight_grad(gc, shape, dtype, layout):
    """Products are exact; a sum of `rows` terms, taken 16 at a time at worst
    with truncation, is off by at most (rows / 16 + 16) 2^-23 of the terms'
    absolute sum."""
    rows, n, k = shape
    ck = gc.ActCheckpoint(rows, k)
    gc.act_compress(matrix(rows, k, "f32", 20), ck)
    dy = matrix(rows, n, dtype, 21, layout, 0.1)
    dy[rows // 2] = 0
    ws = gc.act_weight_grad_workspace(rows, n, k, DT[dtype])
    q, d = read(ck), f64(dy)
    if rows > 1:
        assert np.isfinite(q).all()
    want, size = d.T @ q, np.abs(d).T @ np.abs(q)
    room = (rows / 16 + 16) * 2.0 ** -23
    scale = (1 + 0.2 * torch.randn(k)).to(DT[dtype]).cuda()
    for cs in (None, scale):
        s = 1.0 if cs is None else f64(cs)
        dw = place(torch.full((n, k), 5.0), layout)
        gc.act_weight_grad(dy, ck, dw, ws, col_scale=cs)
        assert (np.abs(f64(dw) - want * s) <= room * size * np.abs(s) + 1e-37).all()
        assert untouched(dw)
        more = torch.full((n, k), 5.0, device="cuda")
        gc.act_weight_grad(dy, ck, more, ws, col_scale=cs, accumulate=True)
        assert (np.abs(f64(more) - 5.0 - want * s) <= room * size * np.abs(s) + 2.0 ** -22 * (5 + np.abs(want))).all()
        again = torch.empty(n, k, device="cuda")
        gc.act_weight_grad(dy, ck, again, ws, col_scale=cs)
        assert torch.equal(again, dw.contiguous())                 # bit-identical from run to run


def test_weight_grad_no_rows(gc):
    ck, dy = gc.ActCheckpoint(0, 40), torch.empty(0, 24, device="cuda", dtype=torch.bfloat16)
    ws = gc.act_weight_grad_workspace(0, 24, 40, torch.bfloat16)
    dw = torch.full((24, 40), 3.0, device="cuda")
    gc.act_weight_grad(dy, ck, dw, ws, accumulate=True)
    assert bool((dw == 3.0).all())
    gc.act_weight_grad(dy, ck, dw, ws)
    assert bool((dw == 0.0).all())


def test_weight_grad_nan_reaches_its_columns_only(gc):
    x = matrix(40, 96, "f32", 22)
    x[7, 40] = float("nan")
    ck, dy = gc.ActCheckpoint(40, 96), matrix(40, 64, "bf16", 23)
    gc.act_compress(x, ck)
    dw = torch.empty(64, 96, device="cuda")
    gc.act_weight_grad(dy, ck, dw, gc.act_weight_grad_workspace(40, 64, 96, torch.bfloat16))
    assert bool(torch.isnan(dw[:, 32:64]).all())                   # the group that holds the NaN
    assert bool(torch.isfinite(dw[:, :32]).all()) and bool(torch.isfinite(dw[:, 64:]).all())


def test_weight_grad_wide_range_of_steps(gc):
    """Steps from 2^-126 to 2^100 in one matrix: every product stays exact."""
    x = matrix(64, 256, "f32", 24, channels=False)
    scale = torch.exp2(torch.linspace(-110, 100, 8)).cuda().repeat_interleave(32)
    x = x * scale
    ck, dy = gc.ActCheckpoint(64, 256), matrix(64, 32, "bf16", 25)
    gc.act_compress(x, ck)
    dw = torch.empty(32, 256, device="cuda")
    gc.act_weight_grad(dy, ck, dw, gc.act_weight_grad_workspace(64, 32, 256, torch.bfloat16))
    want, size = f64(dy).T @ read(ck), np.abs(f64(dy)).T @ np.abs(read(ck))
    assert (np.abs(f64(dw) - want) <= 20 * 2.0 ** -23 * size + 1e-38).all()


# ----------------------------------------------------------------------------- all of it

def test_empty_rows(gc):
    ck = gc.ActCheckpoint(0, 50)
    x = torch.empty(0, 50, device="cuda")
    gc.act_compress(x, ck)
    gc.act_decompress(ck, x)
    gc.rmsnorm(x, None, 1e-5, x.clone(), ckpt=ck)
    dw = torch.full((50,), 2.0, device="cuda")
    ws = gc.rmsnorm_backward_workspace(0, 50)
    gc.rmsnorm_backward(x, ck, torch.empty(0, device="cuda"), None, x.clone(), dw, ws, accumulate=True)
    assert bool((dw == 2.0).all())
    gc.rmsnorm_backward(x, ck, torch.empty(0, device="cuda"), None, x.clone(), dw, ws)
    assert bool((dw == 0.0).all())
    gc.gated_act(0, x, x, x.clone())
    torch.cuda.synchronize()


def test_side_stream_and_graph(gc):
    """Calls follow the stream that they are given, and replay from a graph."""
    x, w = matrix(64, 512, "bf16", 30), torch.ones(512, device="cuda")
    dy = matrix(64, 512, "bf16", 31)
    y, dx, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda")
    dw, dW = torch.empty(512, device="cuda"), torch.empty(512, 512, device="cuda")
    ck = gc.ActCheckpoint(64, 512)
    ws, ws2 = gc.rmsnorm_backward_workspace(64, 512), gc.act_weight_grad_workspace(64, 512, 512, torch.bfloat16)

    def step(stream=None):
        gc.rmsnorm(x, w, 1e-5, y, rstd=rstd, ckpt=ck, stream=stream)
        gc.rmsnorm_backward(dy, ck, rstd, w, dx, dw, ws, stream=stream)
        gc.act_weight_grad(dy, ck, dW, ws2, stream=stream)

    step()
    want = [t.clone() for t in (y, dx, dw, dW)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (y, dx, dw, dW):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    for t, v in zip((y, dx, dw, dW), want):
        assert torch.equal(t, v)
        t.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t in (y, dx, dw, dW):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, v in zip((y, dx, dw, dW), want):
            assert torch.equal(t, v)


def test_guard_bytes(gc):
    """Nothing is written outside codes, steps, vectors and workspaces."""
    rows, cols, n = 9, 100, 70
    ldc = 128

    def guarded(count, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((count * size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[256:256 + count * size].view(dtype)

    x = matrix(rows, cols, "f16", 40)
    bufs = {}
    bufs["codes"], codes = guarded(rows * ldc, torch.int8)
    bufs["steps"], steps = guarded(rows * ldc // 32, torch.uint8)
    bufs["rstd"], rstd = guarded(rows, torch.float32)
    bufs["dw"], dw = guarded(cols, torch.float32)
    bufs["ws"], ws = guarded(gc.rmsnorm_backward_workspace(rows, cols).numel(), torch.uint8)
    bufs["ws2"], ws2 = guarded(gc.act_weight_grad_workspace(rows, n, cols, torch.float16).numel(), torch.uint8)
    bufs["dW"], dW = guarded(n * cols, torch.float32)
    ck = gc.ActCheckpoint(rows, cols, codes=codes.view(rows, ldc), steps=steps.view(rows, ldc // 32))
    y = torch.empty_like(x)
    gc.act_compress(x, ck)
    gc.rmsnorm(x, None, 1e-5, y, rstd=rstd, ckpt=ck)
    gc.rmsnorm_backward(x, ck, rstd, None, y, dw, ws)
    gc.act_weight_grad(matrix(rows, n, "f16", 41), ck, dW.view(n, cols), ws2)
    gc.gated_act(0, x, x, y, ckpt_gate=ck, ckpt_up=gc.ActCheckpoint(rows, cols))
    torch.cuda.synchronize()
    for name, b in bufs.items():
        assert bool((b[:256] == 0xA5).all()) and bool((b[-256:] == 0xA5).all()), name


def test_matrices_beyond_two_to_the_31_elements(gc):
    """Offsets past 32 bits: the last rows of a matrix of 2.2e9 elements give
    what they give on their own."""
    rows, cols, tail = 135000, 16384, 64
    x = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16).normal_()
    ck, small = gc.ActCheckpoint(rows, cols), gc.ActCheckpoint(tail, cols)
    last = x[-tail:]
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")

    def same(big, little):
        return torch.equal(big[-tail:], little)

    gc.act_compress(x, ck)
    gc.act_compress(last, small)
    assert same(ck.codes, small.codes) and same(ck.steps, small.steps)
    y2, rstd2 = torch.empty_like(last), torch.empty(tail, device="cuda")
    gc.act_decompress(ck, y)
    gc.act_decompress(small, y2)
    assert same(y, y2)
    gc.rmsnorm(x, None, 1e-5, y, rstd=rstd, ckpt=ck)
    gc.rmsnorm(last, None, 1e-5, y2, rstd=rstd2, ckpt=small)
    assert same(y, y2) and same(ck.codes, small.codes) and same(rstd, rstd2)
    gc.rmsnorm_backward(x, ck, rstd, None, y, None, None)
    gc.rmsnorm_backward(last, small, rstd2, None, y2, None, None)
    assert same(y, y2)
    gc.gated_act_backward(0, x, ck, ck, y, x)                      # dup over dout
    keep = torch.empty_like(last)
    last2 = torch.empty_like(last)
    torch.cuda.synchronize()
    keep.copy_(y[-tail:])
    del y
    dW, dW2 = torch.empty(16, cols, device="cuda"), torch.empty(16, cols, device="cuda")
    # a gradient that is zero except in the last rows gives those rows' sums
    dy = torch.zeros(rows, 16, device="cuda", dtype=torch.bfloat16)
    dy[-tail:].normal_()
    gc.act_weight_grad(dy, ck, dW, gc.act_weight_grad_workspace(rows, 16, cols, torch.bfloat16))
    gc.act_weight_grad(dy[-tail:], small, dW2, gc.act_weight_grad_workspace(tail, 16, cols, torch.bfloat16))
    scale = dW2.abs().max()
    assert float((dW - dW2).abs().max() / scale) <= (tail / 16 + 16) * 2.0 ** -22
