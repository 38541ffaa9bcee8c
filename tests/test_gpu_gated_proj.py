"""Gated projection and its gradient against plain 64-bit forms.

Tolerances.  Products of 16-bit operands are exact in fp32; the tensor cores
add 16 of them at a time to an accumulator and truncate, an error of at most
2^-22 of the terms' absolute sum S a step (2^-23 for the accumulator's own
truncation, as much again for the alignment of the 16 terms), so a sum over k
terms is within (ceil(k / 16) + 8) 2^-22 S.  What the activation does to that goes
by its slope, at most 1.13, and the activation itself is within 2^-16 of its
value.  The output is the rounding of the result: half a step of its type at the
far end of that interval, and half the smallest number.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
KINDS = ["silu", "gelu"]


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


def kind_of(gc, kind):
    return gc.GC_GATE_SILU if kind == "silu" else gc.GC_GATE_GELU_TANH


def act64(kind, g):
    """act(g) and act'(g) in 64 bits."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    root = math.sqrt(2 / math.pi)
    t = torch.tanh(root * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * root * (1 + 0.134145 * g * g)


def sums64(x, w):
    """x w^T and the bound of its error."""
    x, w = x.double().cpu(), w.double().cpu()
    steps = -(-x.shape[1] // 16) + 8
    return x @ w.T, (x.abs() @ w.abs().T) * steps * 2.0 ** -22


def rounded(value, error, dtype):
    """How far the rounding to dtype of something within `error` of value may be."""
    return error + (value.abs() + error) * (torch.finfo(dtype).eps / 2) + TINY[dtype] / 2


def strided(rows, cols, dtype, ld, off, gen=None, scale=1.0):
    """rows x cols in a buffer of ld columns from column off on; the rest 77."""
    buf = torch.full((rows, ld), 77.0, dtype=dtype, device="cuda")
    view = buf[:, off:off + cols]
    if gen is not None:
        view.copy_((scale * torch.randn(rows, cols, generator=gen)).to(dtype))
    return buf, view


def outside_kept(buf, off, cols):
    keep = torch.ones(buf.shape[1], dtype=torch.bool)
    keep[off:off + cols] = False
    return bool((buf[:, keep.cuda()] == 77.0).all())


def read(ck):
    step = torch.exp2(ck.steps.double().cpu() - 127).repeat_interleave(32, 1)
    return torch.where(ck.steps.cpu().repeat_interleave(32, 1) == 255, float("nan"), ck.codes.double().cpu() * step)


def check_held(ck, value, error):
    """The checkpoint is one of a matrix within `error` of value."""
    rows, cols = value.shape
    ldc = -(-cols // 32) * 32
    pad = torch.nn.functional.pad
    low = pad((value.abs() - error).clamp(min=0), (0, ldc - cols)).view(rows, -1, 32).amax(2)
    high = pad(value.abs() + error, (0, ldc - cols)).view(rows, -1, 32).amax(2)

    def step(top):
        b = torch.frexp(top)[1] - 7
        b = b + (torch.round(top * torch.exp2(-b.double())) > 127).int()
        return torch.where(top == 0, 1, (b + 127).clamp(1, 248))

    got = ck.steps.cpu().int()
    assert bool((got >= step(low)).all()) and bool((got <= step(high)).all())
    half = torch.exp2(got.double() - 128).repeat_interleave(32, 1)[:, :cols]
    assert bool(((read(ck)[:, :cols] - value).abs() <= half * (1 + 2.0 ** -20) + error).all())
    assert int(ck.codes.cpu()[:, cols:].abs().sum()) == 0


# (rows, n, k): one token to several tiles, one stage to several rings, widths around every tile's
SHAPES = [(1, 1, 1), (1, 32, 64), (2, 33, 65), (5, 31, 7), (77, 333, 1001), (128, 128, 128), (129, 257, 320), (1, 4096, 1024),
          (16, 4865, 72), (300, 1000, 264), (1031, 96, 520), (48, 640, 4096), (260, 5000, 136), (3, 70, 520), (4, 4097, 264),
          (30, 1200, 1096), (100, 64, 2000),
          (8, 500, 300), (2, 301, 130), (6, 2000, 1500),
          (40, 129, 64), (100, 129, 64), (9, 1171, 2000), (40, 2344, 4096), (129, 101, 64), (129, 516, 4096), (129, 2515, 520), (300, 4867, 64),
          (2, 300, 8192), (7, 16, 600), (40, 200, 300), (3, 640, 5120), (333, 16, 64), (5, 1, 1025)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(gc, shape, dtype, kind):
    rows, n, k = shape
    dt = DT[dtype]
    gen = torch.Generator().manual_seed(rows * 7919 + n * 31 + k)
    # rows on 16-byte boundaries, then anywhere
    for lds, offs in (((k + 15) // 8 * 8, 8 * ((n + 15) // 8)), (0, 0, 0)), ((k + 3, n + 5), (1, 2, 3)):
        xb, x = strided(rows, k, dt, lds[0], offs[0], gen)
        wb, w = strided(2 * n, k, dt, lds[0], offs[1], gen, k ** -0.5)
        ob, out = strided(rows, n, dt, lds[1], offs[2])
        wg, wu = w[:n], w[n:]
        ws = gc.gated_proj_workspace(x, wg, wu)
        g, dg = sums64(x, wg)
        u, du = sums64(x, wu)
        f, _ = act64(kind, g)
        error = 1.13 * dg * (u.abs() + du) + f.abs() * du + 2.0 ** -16 * (f * u).abs()
        for kept in (False, True):
            cks = [gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)] if kept else [None, None]
            out.fill_(5.0)
            gc.gated_proj(kind_of(gc, kind), x, wg, wu, out, ws, *cks)
            assert gc.get_device_status(ws).error_bits == 0
            off = (out.double().cpu() - f * u).abs()
            assert bool((off <= rounded(f * u, error, dt)).all()), float((off / rounded(f * u, error, dt)).max())
            assert outside_kept(ob, offs[2], n) and outside_kept(xb, offs[0], k) and outside_kept(wb, offs[1], k)
            if kept:
                check_held(cks[0], g, dg)
                check_held(cks[1], u, du)


def test_forward_is_the_same_from_run_to_run_and_layout_to_layout(gc):
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(300, 264, generator=gen).to(torch.bfloat16).cuda()
    w = (torch.randn(2000, 264, generator=gen) / 16).to(torch.bfloat16).cuda()
    ws = gc.gated_proj_workspace(x, w[:1000], w[1000:])
    outs = [torch.empty(300, 1000, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    gc.gated_proj(0, x, w[:1000], w[1000:], outs[0], ws)
    gc.gated_proj(0, x, w[:1000], w[1000:], outs[1], ws)
    xb, xs = strided(300, 264, torch.bfloat16, 271, 3)
    xs.copy_(x)
    gc.gated_proj(0, xs, w[:1000], w[1000:], outs[2], gc.gated_proj_workspace(xs, w[:1000], w[1000:]))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 77, 261), (1, 30, 4099), (3, 129, 300), (5, 33, 2500), (8, 64, 515), (8, 1111, 1301), (40, 129, 67), (9, 1171, 2001), (129, 101, 68)])
def test_what_lies_around_the_matrices_does_not_matter(gc, shape, dtype):
    """Rows on 16-byte boundaries and rows anywhere, between zeros and between NaN: the same bits;
    and a column of weights that is not finite spoils that one alone."""
    rows, n, k = shape
    dt = DT[dtype]
    gen = torch.Generator().manual_seed(rows + n + k)
    x, w = torch.randn(rows, k, generator=gen).to(dt), (torch.randn(2 * n, k, generator=gen) * k ** -0.5).to(dt)

    def run(ld, off, around, w):
        xb, wb = torch.full((rows, ld), around, dtype=dt, device="cuda"), torch.full((2 * n, ld), around, dtype=dt, device="cuda")
        xb[:, off:off + k], wb[:, off:off + k] = x.cuda(), w.cuda()
        xv, wg, wu = xb[:, off:off + k], wb[:n, off:off + k], wb[n:, off:off + k]
        out = torch.empty(rows, n, dtype=dt, device="cuda")
        ws = gc.gated_proj_workspace(xv, wg, wu)
        ws.fill_(255)                                  # NaN, too, in either type
        gc.gated_proj(0, xv, wg, wu, out, ws)
        assert gc.get_device_status(ws).error_bits == 0
        return out.cpu()

    up = (k + 23) // 8 * 8
    want = run(up, 8, 0.0, w)
    assert bool(torch.isfinite(want).all())
    for ld, off in ((up, 8), (up + 3, 1), (k, 0)):
        assert torch.equal(run(ld, off, float("nan"), w), want), (ld, off)
    j = n // 2
    w[j, k - 1] = float("nan")
    for ld, off in ((up, 8), (up + 3, 1)):
        got = run(ld, off, 0.0, w)
        assert bool(torch.isnan(got[:, j]).all())
        got[:, j] = want[:, j]
        assert torch.equal(got, want), (ld, off)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_that_is_not_finite_spoils_no_other(gc, bad):
    """And what is outside the matrices is zero to every row, also to that one's pads."""
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(200, 100, generator=gen).to(torch.float16)
    w = torch.randn(2 * 50, 100, generator=gen).to(torch.float16).cuda() / 8
    clean, out = (torch.empty(200, 50, dtype=torch.float16, device="cuda") for _ in range(2))
    ck = [[gc.ActCheckpoint(200, 50) for _ in range(2)] for _ in range(2)]
    xc = x.cuda()
    ws = gc.gated_proj_workspace(xc, w[:50], w[50:])
    gc.gated_proj(0, xc, w[:50], w[50:], clean, ws, *ck[0])
    x[131, 17] = bad
    gc.gated_proj(0, x.cuda(), w[:50], w[50:], out, ws, *ck[1])
    others = torch.arange(200) != 131
    assert torch.equal(out.cpu()[others], clean.cpu()[others])
    assert not bool(torch.isfinite(out[131]).any()) or bad == float("inf")
    for a, b in zip(*ck):
        assert torch.equal(a.codes.cpu()[others], b.codes.cpu()[others])
        assert bool((b.steps[131] == 255).all()) and int(b.codes[131].abs().sum()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES + [(128, 9000, 64), (40, 14336, 1024), (31, 2100, 96), (600, 8200, 300), (257, 4500, 1001)])
def test_backward(gc, shape, dtype, kind):
    rows, n, k = shape
    dt = DT[dtype]
    gen = torch.Generator().manual_seed(rows * 7 + n * 3 + k)
    cg, cu = gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)
    gc.act_compress(torch.randn(rows, n, generator=gen).cuda(), cg)
    gc.act_compress(torch.randn(rows, n, generator=gen).cuda(), cu)
    for lds, offs in (((n + 15) // 8 * 8, (k + 15) // 8 * 8), (0, 0, 0, 0)), ((2 * n + 9, k + 3), (1, 2, 3, n + 4)):
        db, d = strided(rows, n, dt, lds[0], offs[0], gen, 0.5)
        wb, w = strided(2 * n, k, dt, lds[1], offs[1], gen, n ** -0.5)
        if offs[3]:
            gb, dg = strided(rows, n, dt, lds[0], 1)
            du = gb[:, offs[3]:offs[3] + n]
        else:
            (gb, dg), (ub, du) = strided(rows, n, dt, lds[0], 0), strided(rows, n, dt, lds[0], 0)
        xb, dx = strided(rows, k, dt, lds[1], offs[2])
        ref = [torch.empty(rows, n, dtype=dt, device="cuda") for _ in range(2)]
        again, again_ref = gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)
        gc.gated_act_backward(kind_of(gc, kind), d, cg, cu, *ref, ckpt_out=again_ref)
        ws = gc.gated_proj_backward_workspace(dg, du, w[:n], w[n:])
        dx.fill_(5.0)
        gc.gated_proj_backward(kind_of(gc, kind), d, cg, cu, w[:n], w[n:], dg, du, dx, ws, ckpt_out=again)
        assert gc.get_device_status(ws).error_bits == 0
        assert torch.equal(dg, ref[0]) and torch.equal(du, ref[1])
        assert torch.equal(again.codes, again_ref.codes) and torch.equal(again.steps, again_ref.steps)
        want, error = sums64(torch.cat(ref, 1), w.T)
        off = (dx.double().cpu() - want).abs()
        assert bool((off <= rounded(want, error, dt)).all()), float((off / rounded(want, error, dt)).max())
        assert outside_kept(xb, offs[2], k) and outside_kept(wb, offs[1], k)
        keep = gb.clone()
        keep[:, (1 if offs[3] else 0):][:, :n] = 77.0
        if offs[3]:
            keep[:, offs[3]:offs[3] + n] = 77.0
        assert bool((keep == 77.0).all())
        # without the checkpoint of the activation, the same
        dx2 = torch.empty(rows, k, dtype=dt, device="cuda")
        gc.gated_proj_backward(kind_of(gc, kind), d, cg, cu, w[:n], w[n:], dg, du, dx2, ws)
        assert torch.equal(dx2, dx)


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_against_differences(gc, kind):
    """Along a direction e, (L(x + h e) - L(x - h e)) / 2h of L = sum(out * dout)
    in 64 bits.  G and U are multiples of 1/64 below 1, so that their
    checkpoints hold them exactly; what is left is the rounding of dgate, dup
    and dx, counted from their values, and h^2 L''' / 6."""
    rows, n, k = 40, 96, 64
    gen = torch.Generator().manual_seed(9)
    # one-hot rows of x pick rows of the transposed weights
    x = torch.zeros(rows, k, dtype=torch.float64)
    x[torch.arange(rows), torch.randint(0, k, (rows,), generator=gen)] = 1.0
    w = torch.randint(-63, 64, (2 * n, k), generator=gen).double() / 64
    d = torch.randn(rows, n, generator=gen).to(torch.bfloat16)
    bf = lambda t: t.to(torch.bfloat16).cuda()  # noqa: E731
    wc, xc = bf(w), bf(x)
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    cg, cu = gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)
    gc.gated_proj(kind_of(gc, kind), xc, wc[:n], wc[n:], out, gc.gated_proj_workspace(xc, wc[:n], wc[n:]), cg, cu)
    g, u = x @ w[:n].T, x @ w[n:].T
    assert torch.equal(read(cg)[:, :n], g) and torch.equal(read(cu)[:, :n], u)
    dg, du = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dx = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    gc.gated_proj_backward(kind_of(gc, kind), d.cuda(), cg, cu, wc[:n], wc[n:], dg, du, dx,
                           gc.gated_proj_backward_workspace(dg, du, wc[:n], wc[n:]))
    e = torch.randn(rows, k, generator=gen, dtype=torch.float64)

    def loss(t):
        return (act64(kind, t @ w[:n].T)[0] * (t @ w[n:].T) * d.double()).sum(1)

    h = 1e-5
    slope = (loss(x + h * e) - loss(x - h * e)) / (2 * h)
    got = (dx.double().cpu() * e).sum(1)
    half = torch.finfo(torch.bfloat16).eps / 2
    both = torch.cat((dg, du), 1).double().cpu().abs()
    allowed = 1.01 * half * ((both @ w.abs()) * e.abs()).sum(1) + 1.01 * half * (dx.double().cpu() * e).abs().sum(1) + 1e-6
    assert bool(((got - slope).abs() <= allowed).all())


def test_no_rows(gc):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(40, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.empty(0, 20, dtype=torch.bfloat16, device="cuda")
    ws = gc.gated_proj_workspace(e, w[:20], w[20:])
    gc.gated_proj(0, e, w[:20], w[20:], o, ws, gc.ActCheckpoint(0, 20), gc.ActCheckpoint(0, 20))
    assert gc.get_device_status(ws).error_bits == 0
    ws = gc.gated_proj_backward_workspace(o, o, w[:20], w[20:])
    gc.gated_proj_backward(0, o, gc.ActCheckpoint(0, 20), gc.ActCheckpoint(0, 20), w[:20], w[20:], o, o, e, ws)
    assert gc.get_device_status(ws).error_bits == 0


def test_rows_far_apart(gc):
    """Offsets past 2^31 elements."""
    ld, rows, n, k = (1 << 30) + 8, 4, 40, 72
    gen = torch.Generator().manual_seed(3)
    small = torch.randn(rows, k, generator=gen).to(torch.bfloat16).cuda()
    w = torch.randn(2 * n, k, generator=gen).to(torch.bfloat16).cuda() / 8
    far = torch.empty(3 * ld + 128, dtype=torch.bfloat16, device="cuda")
    x, out = far.as_strided((rows, k), (ld, 1)), far.as_strided((rows, n), (ld, 1), 80)
    x.copy_(small)
    ref = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    ws = gc.gated_proj_workspace(x, w[:n], w[n:])
    gc.gated_proj(0, small, w[:n], w[n:], ref, ws)
    gc.gated_proj(0, x, w[:n], w[n:], out, ws)
    assert torch.equal(out, ref)
    cg, cu = gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)
    gc.gated_proj(0, small, w[:n], w[n:], ref, ws, cg, cu)
    d = torch.randn(rows, n, generator=gen).to(torch.bfloat16).cuda()
    dg, du = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = gc.gated_proj_backward_workspace(dg, du, w[:n], w[n:])
    want, dx = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda"), far.as_strided((rows, k), (ld, 1))
    gc.gated_proj_backward(0, d, cg, cu, w[:n], w[n:], dg, du, want, ws)
    gc.gated_proj_backward(0, d, cg, cu, w[:n], w[n:], dg, du, dx, ws)
    assert torch.equal(dx, want)


def test_streams_and_graphs(gc):
    """On another stream, and captured and replayed with other inputs, beside direct calls."""
    rows, n, k = 130, 200, 328
    gen = torch.Generator().manual_seed(4)
    xs = [torch.randn(rows, k, generator=gen).to(torch.float16).cuda() for _ in range(3)]
    ds = [torch.randn(rows, n, generator=gen).to(torch.float16).cuda() for _ in range(3)]
    w = (torch.randn(2 * n, k, generator=gen) / 16).to(torch.float16).cuda()

    def buffers():
        b = dict(out=torch.empty(rows, n, dtype=torch.float16, device="cuda"), cg=gc.ActCheckpoint(rows, n),
                 cu=gc.ActCheckpoint(rows, n), dg=torch.empty(rows, n, dtype=torch.float16, device="cuda"),
                 du=torch.empty(rows, n, dtype=torch.float16, device="cuda"),
                 dx=torch.empty(rows, k, dtype=torch.float16, device="cuda"))
        b["ws"], b["wb"] = gc.gated_proj_workspace(xs[0], w[:n], w[n:]), gc.gated_proj_backward_workspace(b["dg"], b["du"], w[:n], w[n:])
        return b

    def step(x, d, b, stream=None):
        gc.gated_proj(1, x, w[:n], w[n:], b["out"], b["ws"], b["cg"], b["cu"], stream=stream)
        gc.gated_proj_backward(1, d, b["cg"], b["cu"], w[:n], w[n:], b["dg"], b["du"], b["dx"], b["wb"], stream=stream)

    wanted = []
    for x, d in zip(xs, ds):
        b = buffers()
        step(x, d, b)
        wanted.append([b[key].clone() for key in ("out", "dg", "du", "dx")])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    b = buffers()
    other.wait_stream(torch.cuda.current_stream())
    step(xs[0], ds[0], b, stream=other)
    other.synchronize()
    assert all(torch.equal(b[key], v) for key, v in zip(("out", "dg", "du", "dx"), wanted[0]))
    x, d, b = xs[0].clone(), ds[0].clone(), buffers()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(x, d, b)
    for i in (1, 2, 0):
        x.copy_(xs[i]), d.copy_(ds[i])
        graph.replay()
        apart = buffers()
        step(xs[i], ds[i], apart)
        torch.cuda.synchronize()
        assert all(torch.equal(b[key], v) for key, v in zip(("out", "dg", "du", "dx"), wanted[i]))
        assert all(torch.equal(apart[key], v) for key, v in zip(("out", "dg", "du", "dx"), wanted[i]))


def test_refusals(gc):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(80, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(4, 40, dtype=torch.bfloat16, device="cuda")
    ck = gc.ActCheckpoint(4, 40)
    ws = gc.gated_proj_workspace(x, w[:40], w[40:])
    wb = gc.gated_proj_backward_workspace(out, out, w[:40], w[40:])
    for f in (lambda: gc.gated_proj(0, x, w[:40], w[40:79], out, ws), lambda: gc.gated_proj(0, x, w[:40, :63], w[40:], out, ws),
              lambda: gc.gated_proj(0, x.half(), w[:40], w[40:], out, ws), lambda: gc.gated_proj(0, x, w[:40], w[40:], x, ws),
              lambda: gc.gated_proj(0, x, w[:40], w[40:], out, ws, gc.ActCheckpoint(4, 41), gc.ActCheckpoint(4, 41)),
              lambda: gc.gated_proj(0, x.t(), w[:40], w[40:], out, ws), lambda: gc.gated_proj(0, x, w[:40], w[40:], out, out),
              lambda: gc.gated_proj_backward(0, out, ck, ck, w[:40], w[40:], out, out, out, wb),
              lambda: gc.gated_proj_backward(0, out, ck, ck, w[:39], w[40:], out, out, x, wb),
              lambda: gc.gated_proj_backward(0, out[:3], ck, ck, w[:40], w[40:], out, out, x, wb)):
        with pytest.raises(ValueError):
            f()
    f32 = [t.float() for t in (x, w[:40], w[40:], out)]
    for f in (lambda: gc.gated_proj(0, *f32, ws), lambda: gc.gated_proj(0, x, w[:40], w[40:], out, ws[256:]),
              lambda: gc.gated_proj(0, x, w[:40], w[40:], out, ws, ck), lambda: gc.gated_proj(7, x, w[:40], w[40:], out, ws),
              lambda: gc.gated_proj(0, torch.zeros(4, 65, dtype=torch.bfloat16, device="cuda")[:, 1:], w[:40], w[40:], out, ws)):
        with pytest.raises(gc.GCError):
            f()


def test_against_the_calls_it_stands_for(gc):
    """Where the projections' outputs are exact in 16 bits: the same as a library's product and gated_act."""
    gen = torch.Generator().manual_seed(8)
    rows, n, k = 100, 320, 64
    x = torch.randint(-2, 3, (rows, k), generator=gen).to(torch.bfloat16).cuda()
    w = (torch.randint(-1, 2, (2 * n, k), generator=gen) / 8).to(torch.bfloat16).cuda()
    both = (x.float() @ w.float().T).to(torch.bfloat16)
    assert torch.equal(both.double().cpu(), x.double().cpu() @ w.double().cpu().T)
    for kind in (0, 1):
        cks = [gc.ActCheckpoint(rows, n) for _ in range(4)]
        out, ref = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        gc.gated_act(kind, both[:, :n], both[:, n:], ref, ckpt_gate=cks[0], ckpt_up=cks[1])
        gc.gated_proj(kind, x, w[:n], w[n:], out, gc.gated_proj_workspace(x, w[:n], w[n:]), cks[2], cks[3])
        assert torch.equal(out, ref)
        for a, b in ((0, 2), (1, 3)):
            assert torch.equal(cks[a].codes, cks[b].codes) and torch.equal(cks[a].steps, cks[b].steps)


def test_two_calls_at_once(gc):
    """On two streams, each with a workspace and outputs of its own."""
    gen = torch.Generator().manual_seed(12)
    rows, n, k = 520, 1500, 700
    x = [torch.randn(rows, k, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    w = (torch.randn(2 * n, k, generator=gen) / 27).to(torch.bfloat16).cuda()
    d = torch.randn(rows, n, generator=gen).to(torch.bfloat16).cuda()

    def buffers(i):
        b = dict(out=torch.empty(rows, n, dtype=torch.bfloat16, device="cuda"), c=[gc.ActCheckpoint(rows, n) for _ in range(2)],
                 d=torch.empty(rows, 2 * n, dtype=torch.bfloat16, device="cuda"), dx=torch.empty_like(x[i]))
        b["ws"] = gc.gated_proj_workspace(x[i], w[:n], w[n:])
        b["wb"] = gc.gated_proj_backward_workspace(b["d"][:, :n], b["d"][:, n:], w[:n], w[n:])
        return b

    def step(i, b, s=None):
        gc.gated_proj(0, x[i], w[:n], w[n:], b["out"], b["ws"], *b["c"], stream=s)
        gc.gated_proj_backward(0, d, *b["c"], w[:n], w[n:], b["d"][:, :n], b["d"][:, n:], b["dx"], b["wb"], stream=s)

    apart = [buffers(i) for i in range(2)]
    for i in range(2):
        step(i, apart[i])
    together, streams = [buffers(i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            step(i, together[i], streams[i])
    torch.cuda.synchronize()
    for a, b in zip(apart, together):
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["dx"], b["dx"]) and torch.equal(a["d"], b["d"])
        assert gc.get_device_status(b["ws"]).error_bits == 0 and gc.get_device_status(b["wb"]).error_bits == 0


def test_a_workspace_does_for_fewer_rows_and_again(gc):
    """Kept from a large call for smaller ones, and used by call after call."""
    gen = torch.Generator().manual_seed(13)
    n, k = 333, 201
    w = (torch.randn(2 * n, k, generator=gen) / 14).to(torch.float16).cuda()
    big = torch.randn(700, k, generator=gen).to(torch.float16).cuda()
    ws = gc.gated_proj_workspace(big, w[:n], w[n:])
    for rows in (700, 1, 64, 129, 3, 700):
        out, ref = (torch.empty(rows, n, dtype=torch.float16, device="cuda") for _ in range(2))
        x = big[:rows]
        gc.gated_proj(1, x, w[:n], w[n:], out, ws)
        gc.gated_proj(1, x, w[:n], w[n:], ref, gc.gated_proj_workspace(x, w[:n], w[n:]))
        assert torch.equal(out, ref) and gc.get_device_status(ws).error_bits == 0


def test_strides_of_one_row(gc):
    """A single row of any stride, also of none."""
    gen = torch.Generator().manual_seed(14)
    k, n = 328, 100
    w = (torch.randn(2 * n, k, generator=gen) / 18).to(torch.bfloat16).cuda()
    x = torch.randn(1, k, generator=gen).to(torch.bfloat16).cuda()
    ref = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    gc.gated_proj(0, x, w[:n], w[n:], ref, gc.gated_proj_workspace(x, w[:n], w[n:]))
    for y in (x.as_strided((1, k), (0, 1)), x.as_strided((1, k), (5, 1)), x.as_strided((1, k), (k + 3, 1)), x[0].unsqueeze(0)):
        out = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
        gc.gated_proj(0, y, w[:n], w[n:], out, gc.gated_proj_workspace(y, w[:n], w[n:]))
        assert torch.equal(out, ref)
        ck = [gc.ActCheckpoint(1, n), gc.ActCheckpoint(1, n)]
        gc.gated_proj(0, y, w[:n], w[n:], out, gc.gated_proj_workspace(y, w[:n], w[n:]), *ck)
        assert float((out.float() - ref.float()).abs().max()) <= 2.0 ** -7 * float(ref.abs().max())
    with pytest.raises(ValueError):
        gc.gated_proj(0, x.expand(3, k), w[:n], w[n:], torch.empty(3, n, dtype=torch.bfloat16, device="cuda"),
                      torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


def test_every_cut_of_a_call(gc):
    """Sizes that the rule for tiles, pairs and splits cuts in different ways,
    inputs of small integers, so that every sum is exact and so is every output."""
    gen = torch.Generator().manual_seed(15)
    for rows, n, k in ((1, 8192, 64), (17, 8192, 96), (33, 14336, 32), (64, 4096, 512), (100, 14336, 128), (128, 2048, 256),
                       (130, 4096, 64), (200, 14336, 256), (256, 1000, 1024), (300, 9000, 64), (512, 14336, 128), (700, 2000, 520),
                       (1031, 4100, 1000), (2048, 1024, 1024), (5000, 100, 64), (9000, 64, 40)):
        dt = torch.bfloat16
        dg = torch.randint(-1, 2, (rows, n), generator=gen, dtype=torch.int8).cuda()
        w = torch.randint(-1, 2, (2 * n, k), generator=gen, dtype=torch.int8).cuda()
        # checkpoints for which dgate = 0 and dup = dout / 2 exactly: act(G) = 1/2 is not
        # exact, so the gradient's product is checked on dup alone, with U = 0
        cg, cu = gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)
        gc.act_compress(torch.full((rows, n), 64.0, dtype=dt, device="cuda"), cg)      # act(64) = 64 in silu
        gc.act_compress(torch.zeros(rows, n, dtype=dt, device="cuda"), cu)
        dout, wd = dg.to(dt), w.to(dt)
        a, b, dx = (torch.empty(rows, c, dtype=dt, device="cuda") for c in (n, n, k))
        wb = gc.gated_proj_backward_workspace(a, b, wd[:n], wd[n:])
        gc.gated_proj_backward(gc.GC_GATE_SILU, dout, cg, cu, wd[:n], wd[n:], a, b, dx, wb)
        assert gc.get_device_status(wb).error_bits == 0
        assert int((a != 0).sum()) == 0 and torch.equal(b, 64 * dout)
        want = (64.0 * (dg.double() @ w[n:].double())).to(dt)
        assert torch.equal(dx, want), (rows, n, k)
        # the projections: G = 0 wherever x's columns are, U from small integers
        x = torch.randint(-1, 2, (rows, k), generator=gen, dtype=torch.int8).cuda()
        out = torch.empty(rows, n, dtype=dt, device="cuda")
        cks = [gc.ActCheckpoint(rows, n) for _ in range(2)]
        gc.gated_proj(gc.GC_GATE_SILU, x.to(dt), wd[:n], wd[n:], out, gc.gated_proj_workspace(x.to(dt), wd[:n], wd[n:]), *cks)
        for ck, part in zip(cks, (w[:n], w[n:])):
            full = x.double() @ part.double().T
            ref = gc.ActCheckpoint(rows, n)
            gc.act_compress(full.float(), ref)
            assert torch.equal(ck.codes, ref.codes) and torch.equal(ck.steps, ref.steps), (rows, n, k)


@pytest.mark.parametrize("off", [0, 1])
def test_gradients_over_dout(gc, off):
    """dgate, or dup, may be dout itself, on 16-byte boundaries and off them."""
    rows, n, k = 150, 424, 328
    gen = torch.Generator().manual_seed(16)
    cks = [gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)]
    for c in cks:
        gc.act_compress(torch.randn(rows, n, generator=gen).cuda(), c)
    w = (torch.randn(2 * n, k, generator=gen) / 20).to(torch.bfloat16).cuda()
    d = torch.randn(rows, n, generator=gen).to(torch.bfloat16).cuda()

    def buffer():
        return torch.zeros(rows, n + 8, dtype=torch.bfloat16, device="cuda")[:, off:off + n]

    def call(dout, dg, du):
        dx = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
        gc.gated_proj_backward(0, dout, *cks, w[:n], w[n:], dg, du, dx, gc.gated_proj_backward_workspace(dg, du, w[:n], w[n:]))
        return dg.clone(), du.clone(), dx

    want = call(d, buffer(), buffer())
    for which in (0, 1):
        own, other = buffer(), buffer()
        own.copy_(d)
        got = call(own, own, other) if which == 0 else call(own, other, own)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_matrix_for_both_projections(gc):
    gen = torch.Generator().manual_seed(17)
    for rows in (1, 50, 300):
        x = torch.randn(rows, 96, generator=gen).to(torch.float16).cuda()
        w = (torch.randn(70, 96, generator=gen) / 10).to(torch.float16).cuda()
        out, ref = (torch.empty(rows, 70, dtype=torch.float16, device="cuda") for _ in range(2))
        gc.gated_proj(0, x, w, w, out, gc.gated_proj_workspace(x, w, w))
        both = torch.cat((w, w))
        gc.gated_proj(0, x, both[:70], both[70:], ref, gc.gated_proj_workspace(x, both[:70], both[70:]))
        assert torch.equal(out, ref)


def test_weights_aligned_apart(gc):
    """One of the weights, or one of the gradients, on 16-byte boundaries and the other off them."""
    gen = torch.Generator().manual_seed(18)
    rows, n, k = 200, 104, 136
    x = torch.randn(rows, k, generator=gen).to(torch.bfloat16).cuda()
    wg, wu = ((torch.randn(n, k, generator=gen) / 12).to(torch.bfloat16).cuda() for _ in range(2))
    d = torch.randn(rows, n, generator=gen).to(torch.bfloat16).cuda()
    cks = [gc.ActCheckpoint(rows, n), gc.ActCheckpoint(rows, n)]

    def moved(t, by):
        m = torch.zeros(t.shape[0], t.shape[1] + 8, dtype=t.dtype, device="cuda")[:, by:by + t.shape[1]]
        m.copy_(t)
        return m

    def call(a, b, c, e):
        wg_, wu_ = moved(wg, a), moved(wu, b)
        out, dx = torch.empty_like(d), torch.empty_like(x)
        gc.gated_proj(1, x, wg_, wu_, out, gc.gated_proj_workspace(x, wg_, wu_), *cks)
        dg, du = moved(d, c), moved(d, e)
        gc.gated_proj_backward(1, d, *cks, wg_, wu_, dg, du, dx, gc.gated_proj_backward_workspace(dg, du, wg_, wu_))
        return out, dg.clone(), du.clone(), dx

    want = call(0, 0, 0, 0)
    for cut in ((0, 1, 0, 0), (3, 0, 0, 0), (0, 0, 0, 5), (0, 0, 7, 0), (1, 2, 3, 4)):
        assert all(torch.equal(a, b) for a, b in zip(call(*cut), want)), cut


def test_codes_past_2_31(gc):
    """A checkpoint and an output of more than 2^31 elements, exact sums: the last rows' are right."""
    rows, n, k = 150_016, 14_336, 64
    gen = torch.Generator(device="cuda").manual_seed(19)
    x = torch.randint(-1, 2, (rows, k), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    w = torch.randint(-1, 2, (2 * n, k), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    out, cks = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda"), [gc.ActCheckpoint(rows, n) for _ in range(2)]
    gc.gated_proj(0, x, w[:n], w[n:], out, gc.gated_proj_workspace(x, w[:n], w[n:]), *cks)
    for rows_ in (slice(0, 130), slice(149_760, 150_016)):
        part = x[rows_]
        ref, few = torch.empty(part.shape[0], n, dtype=torch.bfloat16, device="cuda"), [gc.ActCheckpoint(part.shape[0], n) for _ in range(2)]
        gc.gated_proj(0, part, w[:n], w[n:], ref, gc.gated_proj_workspace(part, w[:n], w[n:]), *few)
        assert torch.equal(out[rows_], ref)
        for a, b in zip(cks, few):
            assert torch.equal(a.codes[rows_], b.codes) and torch.equal(a.steps[rows_], b.steps)
    # and its gradient, over the outputs
    d, dx = out, torch.empty_like(x)
    dg = torch.empty_like(out)
    gc.gated_proj_backward(0, d, *cks, w[:n], w[n:], dg, d, dx, gc.gated_proj_backward_workspace(dg, d, w[:n], w[n:]))
    last = slice(149_760, 150_016)
    ck = [gc.ActCheckpoint(256, n, codes=c.codes[last].clone(), steps=c.steps[last].clone()) for c in cks]
    g2, u2, x2 = torch.empty_like(ref), torch.empty_like(ref), torch.empty(256, k, dtype=torch.bfloat16, device="cuda")
    gc.gated_proj_backward(0, ref, *ck, w[:n], w[n:], g2, u2, x2, gc.gated_proj_backward_workspace(g2, u2, w[:n], w[n:]))
    assert torch.equal(dg[last], g2) and torch.equal(d[last], u2)
    want, error = sums64(torch.cat((g2, u2), 1), w.T)
    for got in (dx[last], x2):
        assert bool(((got.double().cpu() - want).abs() <= rounded(want, error, torch.bfloat16)).all())
