"""The gates far out on the left, where their factors leave fp32's normal numbers."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    gcmod.lib()
    return gcmod


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gates_far_out_on_the_left(gc, dtype, kind):
    """The activation and its gradient down to the type's smallest numbers.
    With u = 2^-24: the exponential turns the roundings of its argument (of
    the product with log2 e, and of that constant) into a relative error of at
    most 2 |p| u, |p| <= 110 here; 2^-16 covers it with the few roundings
    around.  Factors below 2^-126 are held to 2^-150, times |g| < 128, and what
    is subtracted in GELU's slope is |p'| < 2^9 times that."""
    far = -110.0 if kind == 0 else -11.0
    g = torch.linspace(far, 0, 4096, device="cuda").to(dtype).view(8, 512)
    u, d = torch.ones_like(g), torch.ones_like(g)
    out, dg, du = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    cg, cu = gc.ActCheckpoint(8, 512), gc.ActCheckpoint(8, 512)
    gc.gated_act(kind, g, u, out, ckpt_gate=cg, ckpt_up=cu)
    gc.gated_act_backward(kind, d, cg, cu, dg, du)
    held, one = torch.empty(8, 512, device="cuda"), torch.empty(8, 512, device="cuda")
    gc.act_decompress(cg, held)
    gc.act_decompress(cu, one)
    assert bool((one == 1).all())

    def act(x):
        x = x.double().cpu().numpy()
        c = 2 * np.sqrt(2 / np.pi)
        p, dp = (x, 1.0) if kind == 0 else (c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x))
        s = 1 / (1 + np.exp(-p))
        return x * s, s, x * s / (1 + np.exp(p)) * dp

    def check(got, want, size):
        room = 2.0 ** -16 * size + 2.0 ** -134
        low, high = (torch.from_numpy(v).to(dtype).double().numpy() for v in (want - room, want + room))
        got = got.double().cpu().numpy()
        bad = ~((low <= got) & (got <= high))
        assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])

    a, _, _ = act(g)
    check(out, a, np.abs(a))
    a, s, rest = act(held)
    check(du, a, np.abs(a))
    check(dg, s + rest, s + np.abs(rest))
