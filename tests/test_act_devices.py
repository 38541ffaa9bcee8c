"""The tensors of an activation call have to be on one GPU (no GPU here: fake
tensors stand for those of two, and no call gets as far as using an address)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


def tensor(gpu, *shape, dtype=torch.bfloat16):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device="cuda:%d" % gpu)


def matrix(gpu):
    return tensor(gpu, 4, 64)


def vector(gpu):
    return tensor(gpu, 64, dtype=torch.float32)


def per_row(gpu):
    return tensor(gpu, 4, dtype=torch.float32)


def space(gpu):
    return tensor(gpu, 1 << 20, dtype=torch.uint8)


def result(gpu):
    return tensor(gpu, 64, 64, dtype=torch.float32)


def kept(gpu):
    import gradient_compression_gb300 as gc
    return gc.ActCheckpoint(4, 64, codes=tensor(gpu, 4, 64, dtype=torch.int8), steps=tensor(gpu, 4, 2, dtype=torch.uint8))


# entry point, its first matrix, the others
CALLS = {
    "act_compress": (lambda gc, x, ckpt: gc.act_compress(x, ckpt, stream=0), [matrix, kept]),
    "act_decompress": (lambda gc, ckpt, out: gc.act_decompress(ckpt, out, stream=0), [kept, matrix]),
    "rmsnorm": (lambda gc, x, w, y, r, h, rstd, ck: gc.rmsnorm(x, w, 1e-5, y, r, h, rstd, ck, stream=0),
                [matrix, vector, matrix, matrix, matrix, per_row, kept]),
    "rmsnorm_backward": (lambda gc, dy, ck, rstd, w, dx, dh: gc.rmsnorm_backward(dy, ck, rstd, w, dx, None, None, dh, stream=0),
                         [matrix, kept, per_row, vector, matrix, matrix]),
    "gated_act": (lambda gc, g, u, o, cg, cu: gc.gated_act(0, g, u, o, cg, cu, stream=0), [matrix, matrix, matrix, kept, kept]),
    "gated_act_backward": (lambda gc, d, cg, cu, dg, du, co: gc.gated_act_backward(0, d, cg, cu, dg, du, co, stream=0),
                           [matrix, kept, kept, matrix, matrix, kept]),
    "act_weight_grad": (lambda gc, dy, ck, dw, ws, cs: gc.act_weight_grad(dy, ck, dw, ws, cs, stream=0),
                        [matrix, kept, result, space, vector]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_one_tensor_elsewhere(gc, name):
    call, makers = CALLS[name]
    for gpu in (0, 1):
        with pytest.raises(gc.GCError):              # all on one: on to the entry point (which finds no address)
            call(gc, *[m(gpu) for m in makers])
        for i in range(len(makers)):
            with pytest.raises(ValueError, match="cuda:[01] where cuda:[01] is needed"):
                call(gc, *[m(gpu ^ (i == j)) for j, m in enumerate(makers)])


def test_arrays_of_a_checkpoint_apart(gc):
    with pytest.raises(ValueError, match="cuda:1 where cuda:0 is needed"):
        gc.ActCheckpoint(4, 64, codes=tensor(0, 4, 64, dtype=torch.int8), steps=tensor(1, 4, 2, dtype=torch.uint8))
