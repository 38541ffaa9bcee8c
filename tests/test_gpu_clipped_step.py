"""The example's training step with clipping: gated projection, its gradient,
the weight gradients, the norm of all of them, clipping, compression."""
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


def run(example, max_norm, steps=1):
    torch.manual_seed(7)
    block = example.GatedBlock(333, 264, 520, density=0.02, seed=5, max_norm=max_norm)
    x, r, dout, dh = (torch.randn(333, 264, device="cuda").to(torch.bfloat16) for _ in range(4))
    block.forward(x, r)
    block.backward(dout, dh)
    whole = block.grad.clone()
    return block, whole, [v.clone() for v in block.compress(0)]


def test_a_clipped_step(example):
    free, whole, sent = run(example, None)
    norm = float(whole.double().norm())
    # the norm is within 18 2^-24 of its value; c and every product round by 2^-24 once more
    tight, same, clipped = run(example, 0.125 * norm)
    assert torch.equal(same, whole)
    assert abs(float(tight.norm) - norm) <= 18 * 2.0 ** -24 * norm
    assert torch.equal(tight.grad, whole * (torch.tensor(0.125 * norm, dtype=torch.float32).cuda() / tight.norm))
    assert abs(float(tight.grad.double().norm()) - 0.125 * norm) <= 21 * 2.0 ** -24 * 0.125 * norm
    assert torch.equal(clipped[0], sent[0])                     # the same entries, as all are scaled alike
    loose, _, untouched = run(example, 2 * norm)
    assert torch.equal(loose.grad, whole)
    assert all(torch.equal(a, b) for a, b in zip(untouched, sent))
