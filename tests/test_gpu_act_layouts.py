"""The activation operators give the same bits whatever the memory layout:
rows on 16-byte boundaries and rows that are not go by different kernels."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    gcmod.lib()
    return gcmod


def off(x):
    """x with rows off every 16-byte boundary."""
    buf = torch.empty(x.shape[0], x.shape[1] + 3, dtype=x.dtype, device=x.device)
    buf[:, 1:-2] = x
    return buf[:, 1:-2]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [1, 33, 500, 512, 513, 1000, 1024, 1030, 2048, 4095, 4096, 5000, 8192, 9000, 16384, 16400, 1500, 2500, 3300, 5120, 12288])
def test_norm(gc, cols, dtype):
    rows = 37
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, r, dy, dh = (torch.randn(rows, cols, generator=gen, device="cuda").to(DT[dtype]) for _ in range(4))
    w = torch.rand(cols, generator=gen, device="cuda").to(DT[dtype])
    got = []
    for place in (lambda t: t, off):
        y, h, dx = (place(torch.empty_like(x)) for _ in range(3))
        rstd, ck = torch.empty(rows, device="cuda"), gc.ActCheckpoint(rows, cols)
        gc.rmsnorm(place(x), w, 1e-5, y, residual=place(r), h=h, rstd=rstd, ckpt=ck)
        gc.rmsnorm_backward(place(dy), ck, rstd, w, dx, None, None, dh=place(dh))
        got.append((y, h, rstd, ck.codes, ck.steps, dx))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [1, 33, 1000, 4096])
def test_gated(gc, cols, dtype, kind):
    rows = 37
    gen = torch.Generator(device="cuda").manual_seed(cols)
    g, u, d = (2 * torch.randn(rows, cols, generator=gen, device="cuda").to(DT[dtype]) for _ in range(3))
    got = []
    for place in (lambda t: t, off):
        a, dg, du, back = (place(torch.empty_like(g)) for _ in range(4))
        cg, cu, ca = (gc.ActCheckpoint(rows, cols) for _ in range(3))
        gc.gated_act(kind, place(g), place(u), a, ckpt_gate=cg, ckpt_up=cu)
        gc.gated_act_backward(kind, place(d), cg, cu, dg, du, ckpt_out=ca)
        gc.act_decompress(ca, back)
        got.append((a, dg, du, back, ca.codes, ca.steps, cg.codes, cu.codes))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [300, 700, 1500, 2500, 3300, 5120, 6001, 9000, 12288])
def test_norm_gradient_against_64_bits(gc, cols, dtype):
    """Every number of warps per row and of rows per CTA.  With u = 2^-24: a sum
    of n products, in any order, is within n u of the sum of their magnitudes;
    dx has a handful of further roundings, and one to its type."""
    rows, u = 700, 2.0 ** -24
    own = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    gen = torch.Generator(device="cuda").manual_seed(cols)
    ck = gc.ActCheckpoint(rows, cols)
    gc.act_compress(torch.randn(rows, cols, generator=gen, device="cuda"), ck)
    dy, dh = (torch.randn(rows, cols, generator=gen, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(cols, generator=gen, device="cuda").to(dtype)
    rstd = 0.5 + torch.rand(rows, generator=gen, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(cols, device="cuda")
    gc.rmsnorm_backward(dy, ck, rstd, w, dx, dw, gc.rmsnorm_backward_workspace(rows, cols), dh=dh)
    q = torch.empty(rows, cols, device="cuda")
    gc.act_decompress(ck, q)
    q, d, gw, r = q.double(), dy.double(), dy.double() * w.double(), rstd.double()[:, None]
    assert ((dw.double() - (d * q).sum(0)).abs() <= (rows + 2) * u * (d * q).abs().sum(0)).all()
    want = r * (gw - q * (gw * q).mean(1, keepdim=True)) + dh.double()
    size = r * (gw.abs() + q.abs() * (gw * q).abs().mean(1, keepdim=True)) + dh.double().abs()
    room = (cols + 8) * u * r * q.abs() * (gw * q).abs().mean(1, keepdim=True) + 8 * u * size
    # fp16 rounds results below 2^-14 to multiples of 2^-24
    assert ((dx.double() - want).abs() <= room + own * (want.abs() + room) + (2.0 ** -25 if dtype == torch.float16 else 0)).all()
