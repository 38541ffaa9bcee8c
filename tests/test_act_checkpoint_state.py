"""The activation calls take a checkpoint's arrays as they are at the call, and
check them then (no GPU: fake tensors stand for CUDA ones, and no call gets as
far as using an address)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


def cuda(*shape, dtype=torch.bfloat16):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device="cuda:0")


def arrays(rows, cols):
    groups = (cols + 31) // 32
    return dict(codes=cuda(rows, 32 * groups, dtype=torch.int8), steps=cuda(rows, groups, dtype=torch.uint8))


def calls(gc, ck):
    """Every call that takes a checkpoint, with ck in each of its places."""
    t, v, rstd, w32 = cuda(4, 64), cuda(64, dtype=torch.float32), cuda(4, dtype=torch.float32), cuda(64, 64, dtype=torch.float32)
    ws = cuda(1 << 20, dtype=torch.uint8)
    good = lambda: gc.ActCheckpoint(4, 64, **arrays(4, 64))                                      # noqa: E731
    return [lambda: gc.act_compress(t, ck, stream=0), lambda: gc.act_decompress(ck, t, stream=0),
            lambda: gc.rmsnorm(t, None, 1e-5, t, ckpt=ck, stream=0),
            lambda: gc.rmsnorm_backward(t, ck, rstd, None, t, v, ws, stream=0),
            lambda: gc.gated_act(0, t, t, t, ckpt_gate=ck, ckpt_up=good(), stream=0),
            lambda: gc.gated_act(0, t, t, t, ckpt_gate=good(), ckpt_up=ck, stream=0),
            lambda: gc.gated_act_backward(0, t, ck, good(), t, t, stream=0),
            lambda: gc.gated_act_backward(0, t, good(), ck, t, t, stream=0),
            lambda: gc.gated_act_backward(0, t, good(), good(), t, t, ckpt_out=ck, stream=0),
            lambda: gc.act_weight_grad(t, ck, w32, ws, stream=0)]


def on_the_host(ck):
    ck.codes = torch.zeros(4, 64, dtype=torch.int8)


def steps_on_the_host(ck):
    ck.steps = torch.zeros(4, 2, dtype=torch.uint8)


def fewer_rows(ck):
    ck.codes = arrays(3, 64)["codes"]


def more_rows(ck):
    ck.rows = 4000


def more_columns(ck):
    ck.cols = 4096


def other_type(ck):
    ck.codes = cuda(4, 64)


def transposed(ck):
    ck.codes = cuda(64, 4, dtype=torch.int8).t()


def gone(ck):
    del ck.codes


def no_tensor(ck):
    ck.steps = 0x10000


@pytest.mark.parametrize("change", [on_the_host, steps_on_the_host, fewer_rows, more_rows, more_columns, other_type,
                                    transposed, gone, no_tensor])
def test_changed_since_it_was_made(gc, change):
    ck = gc.ActCheckpoint(4, 64, **arrays(4, 64))
    for f in calls(gc, ck):
        with pytest.raises(gc.GCError):              # as it should be: on to the entry point (which finds no address)
            f()
    change(ck)
    for f in calls(gc, ck):
        with pytest.raises(ValueError):
            f()


def test_size_raised_with_the_matrix(gc):
    """The arrays are checked against the checkpoint's size, too."""
    for rows, cols in ((4000, 64), (4, 4096)):
        ck, t = gc.ActCheckpoint(4, 64, **arrays(4, 64)), cuda(rows, cols)
        ck.rows, ck.cols = rows, cols
        for f in (lambda: gc.act_compress(t, ck, stream=0), lambda: gc.act_decompress(ck, t, stream=0),
                  lambda: gc.rmsnorm(t, None, 1e-5, t, ckpt=ck, stream=0),
                  lambda: gc.gated_act_backward(0, t, ck, ck, t, t, stream=0)):
            with pytest.raises(ValueError):
                f()


def test_not_a_checkpoint(gc):
    class Numbers:
        rows, cols, _codes, _steps = 4, 64, 0x10000, 0x10000

    for ck in (Numbers, 3, "x", arrays(4, 64)["codes"]):
        for f in calls(gc, ck):
            with pytest.raises(ValueError):
                f()
