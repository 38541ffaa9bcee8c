"""Arguments of the activation and gradient calls that are easily taken for others."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


@pytest.mark.parametrize("kind", [2, -1, 1 << 32, (1 << 32) + 1, -(1 << 32), 1 << 40])
def test_no_kind_of_activation(gc, kind):
    """Also where its lower 32 bits are one."""
    rows, n, k = 4, 64, 32
    x, w = torch.ones(rows, k, device="cuda").bfloat16(), torch.ones(2 * n, k, device="cuda").bfloat16()
    gate, out, d, dx = (torch.full((rows, c), 7.0, device="cuda").bfloat16() for c in (n, n, n, k))
    cks = [gc.ActCheckpoint(rows, n) for _ in range(2)]
    for c in cks:
        gc.act_compress(gate, c)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for call in (lambda: gc.gated_act(kind, gate, gate, out), lambda: gc.gated_act_backward(kind, gate, *cks, out, d),
                 lambda: gc.gated_proj(kind, x, w[:n], w[n:], out, ws),
                 lambda: gc.gated_proj_backward(kind, gate, *cks, w[:n], w[n:], out, d, dx, gc.gated_proj_backward_workspace(out, d, w[:n], w[n:]))):
        with pytest.raises(gc.GCError):
            call()
    assert all(bool((t == 7.0).all()) for t in (out, d, dx))
