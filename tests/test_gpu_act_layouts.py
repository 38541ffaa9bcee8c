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
@pytest.mark.parametrize("cols", [1, 33, 500, 512, 513, 1000, 1024, 1030, 2048, 4095, 4096, 5000, 8192, 9000, 16384, 16400])
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
