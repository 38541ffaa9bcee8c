"""The compiled argument marshalling of the activation operators: what it
refuses without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


class Kept:
    """A checkpoint's size and addresses; no call below gets as far as using them."""
    rows, cols, _codes, _steps = 4, 64, 0x10000, 0x10000


def calls(gc, t):
    """Every entry point with t as its leading matrix."""
    return {"act_compress": lambda: gc.act_compress(t, Kept), "act_decompress": lambda: gc.act_decompress(Kept, t),
            "rmsnorm": lambda: gc.rmsnorm(t, None, 1e-5, t),
            "rmsnorm_backward": lambda: gc.rmsnorm_backward(t, Kept, t, None, t, None, None),
            "gated_act": lambda: gc.gated_act(0, t, t, t),
            "gated_act_backward": lambda: gc.gated_act_backward(0, t, Kept, Kept, t, t),
            "act_weight_grad": lambda: gc.act_weight_grad(t, Kept, t, t)}


@pytest.mark.parametrize("what", [torch.zeros(4, 64), torch.zeros(4), torch.zeros(()), torch.zeros(4, 64, dtype=torch.int32),
                                  None, 3.0, "x"])
def test_not_a_cuda_matrix(gc, what):
    for name, f in calls(gc, what).items():
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("shape", [(-1, 64), (4, 0)])
def test_checkpoint_shape(gc, shape):
    with pytest.raises(ValueError):
        gc.ActCheckpoint(*shape, device="cpu")


def test_checkpoint_arrays(gc):
    codes, steps = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    for c, s in ((codes, steps), (codes.int(), steps), (codes, steps[:, :1]), (codes.t(), steps), (codes, "x")):
        with pytest.raises(ValueError):                  # no CUDA tensors, or worse
            gc.ActCheckpoint(4, 64, codes=c, steps=s)


def test_number_of_arguments(gc):
    from gradient_compression_gb300 import _marshal, activations
    activations._marshal()
    with pytest.raises(TypeError):
        _marshal.rmsnorm(1, 2)
    with pytest.raises(TypeError):
        _marshal.bind(1)
