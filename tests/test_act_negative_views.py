"""Views that PyTorch keeps as the negative of their memory (the imaginary part
of a conjugate) are refused: what the kernels read there has the other sign."""
import pytest
import torch


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


def test_refused_before_anything_else(gc):
    z = torch.ones(4, 1, dtype=torch.complex64)
    t = z.conj().imag
    assert t.is_neg() and float(t[0]) == 0.0
    v = t[:1, 0]                                                    # a dense one
    ws, plain = torch.zeros(256, dtype=torch.uint8), torch.zeros(1)
    for call in (lambda: gc.grad_norm([plain], v, ws), lambda: gc.grad_clip([plain], v, 1.0), lambda: gc.rmsnorm(t, None, 1e-5, t),
                 lambda: gc.gated_act(0, t, t, t), lambda: gc.gated_proj(0, t, t, t, t, ws),
                 lambda: gc.act_weight_grad(t, None, t, ws), lambda: gc.act_decompress(None, t)):
        with pytest.raises(ValueError, match="sign"):
            call()


@pytest.mark.gpu
def test_refused_in_lists(gc, cuda_device):
    v = torch.full((1,), 1 + 2j, dtype=torch.complex64, device="cuda").conj().imag
    assert v.is_neg() and float(v) == -2.0
    norm, out = torch.tensor([4.0], device="cuda"), torch.full((1,), 7.0, device="cuda")
    for call in (lambda: gc.grad_norm([v], out, gc.grad_norm_workspace([v])), lambda: gc.grad_clip([v], norm, 2.0, out=[out]),
                 lambda: gc.grad_clip([out], norm, 2.0, out=[v]), lambda: gc.grad_clip([v], norm, 2.0)):
        with pytest.raises(ValueError, match="sign"):
            call()
    assert float(out) == 7.0
    gc.grad_clip([v.resolve_neg()], norm, 2.0, out=[out])
    assert float(out) == -1.0
