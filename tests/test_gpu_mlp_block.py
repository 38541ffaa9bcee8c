"""The example's training step: every activation operator together, and the
compressor on what they put into the arena."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import mlp_block
    return mlp_block


def reference(block, x, r, dout, dh, eps):
    """Gradients of the same block in 64 bits, activations kept whole."""
    w, wgu, wd = (t.double().requires_grad_() for t in (block.w, block.wgu, block.wd))
    x = x.double().requires_grad_()
    h = x + r.double()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + eps) * w
    g, u = (y @ wgu.T).split(block.hidden, 1)
    out = (torch.nn.functional.silu(g) * u) @ wd.T
    ((out * dout.double()).sum() + (h * dh.double()).sum()).backward()
    return out.detach(), x.grad, wgu.grad, wd.grad, w.grad


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("shape", [(300, 256, 520), (1024, 512, 1024)])
def test_gradients_of_a_step(example, shape):
    """A value held in 8 bits is off by at most half a step, 1/127 of its
    group's largest magnitude, as if uniform: 1/220 of it in the mean square,
    about 1.5% of a value where the largest is three times the usual one.  The
    products round to bf16 (2^-9) on top; 4% of a gradient's norm covers both
    for gradients that pass two of the checkpoints."""
    tokens, width, hidden = shape
    block = example.GatedBlock(tokens, width, hidden, seed=3)
    block.w += 0.1 * torch.randn(width, device="cuda")
    x, r, dout, dh = (torch.randn(tokens, width, device="cuda").to(torch.bfloat16) for _ in range(4))
    out, h = block.forward(x, r)
    dx = block.backward(dout, dh).clone()
    want = reference(block, x, r, dout, dh, example.EPS)
    assert off(out, want[0]) < 0.02
    assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16))
    for got, ref in ((dx, want[1]), (block.dwgu, want[2]), (block.dwd, want[3]), (block.dw, want[4])):
        assert off(got, ref) < 0.04
    once = block.grad.clone()
    block.backward(dout, dh, accumulate=True)                      # a second micro-batch of the same
    assert off(block.grad, 2 * once.double()) < 1e-5
    assert block.kept_bytes < 0.36 * 2 * tokens * (2 * width + 3 * hidden)


def test_compression_of_the_arena(example):
    """The compressor's payload and residual add up to the arena exactly."""
    block = example.GatedBlock(256, 256, 512, density=0.05, seed=4)
    x, r, dout, dh = (torch.randn(256, 256, device="cuda").to(torch.bfloat16) for _ in range(4))
    block.forward(x, r)
    block.backward(dout, dh)
    idx, q, scale = block.compress(0)
    import gradient_compression_gb300 as gc
    assert gc.get_device_status(block.compressor.workspace).error_bits == 0
    off_, koff = block.layout.off, block.layout.koff
    for t in range(block.layout.T):
        e = block.error[off_[t]:off_[t + 1]]
        g = block.grad[off_[t]:off_[t + 1]]
        i = idx[koff[t]:koff[t + 1]].long()
        assert bool((i[1:] > i[:-1]).all())
        sent = torch.zeros_like(g)
        sent[i] = q[koff[t]:koff[t + 1]].float() * scale[t]
        assert torch.equal(e, g - sent)
        kept = g[i].abs().min()
        rest = torch.ones_like(g, dtype=torch.bool)
        rest[i] = False
        assert float(g[rest].abs().max()) <= float(kept)


def test_command_line(example, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["mlp_block.py", "--tokens", "64", "--width", "128", "--hidden", "256", "--steps", "2"])
    example.main()
    out = capsys.readouterr().out
    assert "step 1" in out and "kept for backward" in out
