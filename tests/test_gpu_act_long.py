"""The activation operators over many rows: what a CTA carries from one of its
tiles, chains or rows to the next.

Weight gradient.  152 CTAs take a matrix's tiles in turn, and a sum over rows
is cut into chains of at most 3200 rows, of which an accumulator's first may be
shorter.  Tolerance: products are exact; a chain adds them up 16 rows at a time
at worst, each addition truncated (2^-23 of what the chain's terms add up to in
size), and the chains' sums are added with one rounding each.  With S the sum
of the terms' sizes the result is within
    (min(rows, 3200) / 16 + 16 + rows / 1600 + splits) 2^-23 S,
far below what a lost or repeated chain, tile or term would change.

The streaming kernels work on a row on its own, so a matrix gives the bits that
its rows give in short pieces (whose values the tests of short matrices hold
against 64 bits): a CTA gets one step of a piece, many of the matrix.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LAYOUTS = ["plain", "odd"]


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    gcmod.lib()
    return gcmod


def place(x, layout):
    """x, or x with rows off every 16-byte boundary, each row differently."""
    if layout == "plain":
        return x
    buf = torch.full((x.shape[0], x.shape[1] + 3), 77.0, dtype=x.dtype, device=x.device)
    buf[:, 1:-2] = x
    return buf[:, 1:-2]


def untouched(view):
    buf = view._base
    return buf is None or bool((buf[:, 0] == 77.0).all() and (buf[:, -2:] == 77.0).all())


def normal(gen, rows, cols, dtype, size=1.0):
    return (size * torch.randn(rows, cols, generator=gen, device="cuda")).to(DT[dtype])


# ------------------------------------------------------------------------ weight gradient

# rows, n, k, type: tiles of 256 x 256 (bf16) or 128 x 256
LONG = [
    (200, 4100, 4100, "bf16"),       # 289 tiles, the last ones of both sides cut
    (300, 4096, 2568, "bf16"),       # 176 tiles, dy copied as it lies (or, odd, loaded by the unpacking warps)
    (200, 2100, 2600, "f16"),        # 187 tiles
    (200, 2100, 2600, "f32"),
    (7000, 2600, 2600, "bf16"),      # 121 tiles, chains in both accumulators
    (7000, 2560, 2568, "bf16"),      # 110 tiles
    (7000, 4096, 2600, "bf16"),      # 176 tiles, and chains
    (7000, 1300, 2600, "f16"),       # 121 tiles, chains of two and of three terms
    (7000, 1300, 2600, "f32"),
    (20000, 1500, 2600, "bf16"),     # 66 tiles, the rows in two parts of several chains each
]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", LONG, ids=lambda c: "%dx%dx%d-%s" % c)
def test_weight_grad(gc, case, layout):
    rows, n, k, dtype = case
    gen = torch.Generator(device="cuda").manual_seed(rows + n)
    ck = gc.ActCheckpoint(rows, k)
    gc.act_compress(normal(gen, rows, k, "f32"), ck)
    dy = place(normal(gen, rows, n, dtype, 0.1), layout)
    q = torch.empty(rows, k, device="cuda")
    gc.act_decompress(ck, q)
    want, size = dy.double().T @ q.double(), dy.double().abs().T @ q.double().abs()
    room = (min(rows, 3200) / 16 + 16 + rows / 1600 + 152) * 2.0 ** -23
    ws = gc.act_weight_grad_workspace(rows, n, k, DT[dtype])
    scale = (1 + 0.2 * torch.randn(k, generator=gen, device="cuda")).to(DT[dtype])
    for cs in (None, scale):
        s = 1.0 if cs is None else cs.double()
        dw = place(torch.full((n, k), 5.0, device="cuda"), layout)
        gc.act_weight_grad(dy, ck, dw, ws, col_scale=cs)
        # two roundings more for the scale
        off = (dw.double() - want * s).abs() - (room + 2.0 ** -23) * size * (abs(s) if cs is None else s.abs())
        assert float(off.max()) <= 0
        assert untouched(dw)
        again = place(torch.full((n, k), 5.0, device="cuda"), layout)
        gc.act_weight_grad(dy, ck, again, ws, col_scale=cs)
        assert torch.equal(again, dw)                              # the same bits from run to run
        # added to what is there: one rounding of numbers up to 5 + |sum| for each chain
        more = place(torch.full((n, k), 5.0, device="cuda"), layout)
        gc.act_weight_grad(dy, ck, more, ws, col_scale=cs, accumulate=True)
        off = (more.double() - 5.0 - want * s).abs() - (room + 2.0 ** -23) * size * (abs(s) if cs is None else s.abs())
        off -= (rows / 1600 + 2) * 2.0 ** -24 * (5.0 + size * (abs(s) if cs is None else s.abs()))
        assert float(off.max()) <= 0
        assert untouched(more)


# -------------------------------------------------------------------- streaming kernels

# Narrow, wide with a cut last group, and whole lines of 16-bit types.
ROWS = [(50000, 34), (3000, 4097), (3000, 2048)]
PIECE = 250


def pieces(rows):
    return [slice(i, min(i + PIECE, rows)) for i in range(0, rows, PIECE)]


def part(gc, ck, s):
    return gc.ActCheckpoint(s.stop - s.start, ck.cols, codes=ck.codes[s], steps=ck.steps[s])


def copy_of(gc, ck):
    new = gc.ActCheckpoint(ck.rows, ck.cols)
    new.codes.fill_(-1)
    new.steps.fill_(17)
    return new


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", ROWS)
def test_checkpoint(gc, shape, dtype, layout):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = place(normal(gen, *shape, dtype), layout)
    ck = gc.ActCheckpoint(*shape)
    small, out, out2 = copy_of(gc, ck), place(torch.zeros_like(x), layout), place(torch.zeros_like(x), layout)
    gc.act_compress(x, ck)
    gc.act_decompress(ck, out)
    for s in pieces(shape[0]):
        gc.act_compress(x[s], part(gc, small, s))
        gc.act_decompress(part(gc, small, s), out2[s])
    assert torch.equal(ck.codes, small.codes) and torch.equal(ck.steps, small.steps)
    assert torch.equal(out, out2) and untouched(out)
    # and the definition: within half a step of every value, which is exact in x's type
    step = torch.exp2(ck.steps.double() - 127).repeat_interleave(32, 1)[:, :shape[1]]
    read = ck.codes.double()[:, :shape[1]] * step
    assert bool(((read - x.double()).abs() <= 0.5 * step).all())
    assert torch.equal(out, read.to(DT[dtype]))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", ROWS)
def test_gated(gc, shape, dtype, layout, kind):
    gen = torch.Generator(device="cuda").manual_seed(2)
    g, u, d = (place(normal(gen, *shape, dtype, 2.0), layout) for _ in range(3))
    got = []
    for whole in (True, False):
        a, dg, du = (place(torch.zeros_like(g), layout) for _ in range(3))
        cg, cu, ca = (copy_of(gc, gc.ActCheckpoint(*shape)) for _ in range(3))
        for s in [slice(0, shape[0])] if whole else pieces(shape[0]):
            pg, pu, pa = (part(gc, c, s) for c in (cg, cu, ca))
            gc.gated_act(kind, g[s], u[s], a[s], ckpt_gate=pg, ckpt_up=pu)
            gc.gated_act_backward(kind, d[s], pg, pu, dg[s], du[s], ckpt_out=pa)
        assert untouched(a) and untouched(dg) and untouched(du)
        got.append((a, dg, du, cg.codes, cg.steps, cu.codes, cu.steps, ca.codes, ca.steps))
    for x, y in zip(*got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(20000, 34), (12000, 700), (6000, 4097), (6000, 2048), (3000, 9001)])
def test_norm(gc, shape, dtype, layout):
    rows, cols = shape
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, r, dy, dh = (place(normal(gen, rows, cols, dtype), layout) for _ in range(4))
    w = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(DT[dtype])
    got = []
    for whole in (True, False):
        y, h, dx = (place(torch.zeros_like(x), layout) for _ in range(3))
        rstd, ck = torch.zeros(rows, device="cuda"), copy_of(gc, gc.ActCheckpoint(rows, cols))
        for s in [slice(0, rows)] if whole else pieces(rows):
            p = part(gc, ck, s)
            gc.rmsnorm(x[s], w, 1e-5, y[s], residual=r[s], h=h[s], rstd=rstd[s], ckpt=p)
            gc.rmsnorm_backward(dy[s], p, rstd[s], w, dx[s], None, None, dh=dh[s])
        assert untouched(y) and untouched(h) and untouched(dx)
        got.append((y, h, dx, rstd, ck.codes, ck.steps))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # dw: a sum of `rows` products in fp32, in any order
    dw = torch.empty(cols, device="cuda")
    gc.rmsnorm_backward(dy, ck, rstd, w, dx, dw, gc.rmsnorm_backward_workspace(rows, cols), dh=dh)
    q = torch.empty(rows, cols, device="cuda")
    gc.act_decompress(ck, q)
    terms = dy.double() * q.double()
    assert bool(((dw.double() - terms.sum(0)).abs() <= (rows + 2) * 2.0 ** -24 * terms.abs().sum(0)).all())
    assert torch.equal(dx, got[0][2])


def test_gated_backward_beyond_two_to_the_31_elements(gc):
    """The last rows of a matrix of 2.2e9 elements, dup over dout."""
    rows, cols, tail = 135000, 16384, 64
    d = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16).normal_()
    ck, small = gc.ActCheckpoint(rows, cols), gc.ActCheckpoint(tail, cols)
    gc.act_compress(d, ck)
    gc.act_compress(d[-tail:], small)
    keep = d[-tail:].clone()
    dg, dg2, du2 = torch.empty_like(d), torch.empty_like(keep), torch.empty_like(keep)
    gc.gated_act_backward(0, keep, small, small, dg2, du2)
    gc.gated_act_backward(0, d, ck, ck, dg, d)
    assert torch.equal(dg[-tail:], dg2) and torch.equal(d[-tail:], du2)
