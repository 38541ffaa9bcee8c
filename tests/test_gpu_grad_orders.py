"""Clipping into tensors of the same shape whose elements lie in the same order,
also where strides of dimensions of one element differ."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


def test_strides_of_single_elements_mean_nothing(gc):
    norm = torch.tensor([4.0], device="cuda")
    base = torch.arange(1.0, 1 + 3 * 5 * 7 * 2, device="cuda").view(2, 5, 7, 3)
    grad = base[:1].permute(0, 3, 1, 2)                                     # (1, 3, 5, 7), channels last
    for first in (5 * 7 * 3, 2 * 5 * 7 * 3, 1, 10 ** 6):
        out = torch.full((5 * 7 * 3 + 8,), 77.0, device="cuda")
        view = out.as_strided((1, 3, 5, 7), (first, 1, 21, 3))
        gc.grad_clip([grad], norm, 2.0, out=[view])
        assert torch.equal(view, grad * 0.5) and bool((out[105:] == 77.0).all())


def test_other_orders_are_refused(gc):
    norm = torch.tensor([4.0], device="cuda")
    grad = torch.ones(1, 3, 5, 7, device="cuda").contiguous(memory_format=torch.channels_last)
    for out in (torch.empty(1, 3, 5, 7, device="cuda"), torch.empty(1, 3, 7, 5, device="cuda").transpose(2, 3),
                torch.empty(1, 5, 3, 7, device="cuda").contiguous(memory_format=torch.channels_last), torch.empty(104, device="cuda")):
        out.fill_(7.0)
        with pytest.raises(ValueError):
            gc.grad_clip([grad], norm, 2.0, out=[out])
        assert bool((out == 7.0).all())


def test_nothing_in_any_order(gc):
    norm = torch.tensor([4.0], device="cuda")
    gc.grad_clip([torch.empty(0, 3, 2, device="cuda").permute(2, 0, 1)], norm, 2.0, out=[torch.empty(0, device="cuda")])
