"""What the activation calls find at the call: a checkpoint where its arrays are
then, a workspace that was set aside for another batch; and what a weight
gradient leaves there for the status call."""
import copy

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


def test_checkpoint_restored_from_the_host(gc):
    """A checkpoint offloaded and brought back to other memory is read there."""
    x = torch.randn(9, 100, device="cuda")
    ck, want, out = gc.ActCheckpoint(9, 100), torch.empty_like(x), torch.empty_like(x)
    gc.act_compress(x, ck)
    gc.act_decompress(ck, want)
    codes, steps = ck.codes, ck.steps                       # the first memory stays alive, and changes
    away = codes.cpu(), steps.cpu()
    ck.codes, ck.steps = away[0].cuda(), away[1].cuda()
    codes.zero_()
    gc.act_decompress(ck, out)
    assert torch.equal(out, want)
    gc.act_compress(2 * x, ck)                              # written there, too
    assert bool((codes == 0).all()) and bool((ck.steps.int() == steps.int() + 1).all())


def test_deep_copy_of_a_checkpoint(gc):
    x = torch.randn(9, 100, device="cuda")
    ck, want, out = gc.ActCheckpoint(9, 100), torch.empty_like(x), torch.empty_like(x)
    gc.act_compress(x, ck)
    gc.act_decompress(ck, want)
    twin = copy.deepcopy(ck)
    gc.act_compress(torch.zeros_like(x), ck)
    gc.act_decompress(twin, out)
    assert torch.equal(out, want)


def test_storage_given_up_and_taken_again(gc):
    """Its memory freed between forward and backward, as sharding and offloading
    do: refused meanwhile, right after."""
    x = torch.randn(9, 100, device="cuda")
    ck, want, out = gc.ActCheckpoint(9, 100), torch.empty_like(x), torch.empty_like(x)
    gc.act_compress(x, ck)
    gc.act_decompress(ck, want)
    away, size = ck.codes.cpu(), ck.codes.untyped_storage().nbytes()
    ck.codes.untyped_storage().resize_(0)
    with pytest.raises(gc.GCError):
        gc.act_decompress(ck, out)
    other = torch.full((size,), 3, dtype=torch.int8, device="cuda")      # somebody else's by now
    ck.codes.untyped_storage().resize_(size)
    ck.codes.copy_(away)
    gc.act_decompress(ck, out)
    assert torch.equal(out, want) and bool((other == 3).all())


def test_weight_grad_of_a_shorter_batch(gc):
    """In the workspace of the full one, which is split into fewer parts."""
    n = k = 512
    ws = gc.act_weight_grad_workspace(16384, n, k, torch.bfloat16)
    for rows in (16384, 16128, 4000, 1):
        ck, dy = gc.ActCheckpoint(rows, k), torch.ones(rows, n, device="cuda", dtype=torch.bfloat16)
        gc.act_compress(torch.ones(rows, k, device="cuda"), ck)
        dw = torch.empty(n, k, device="cuda")
        gc.act_weight_grad(dy, ck, dw, ws)
        assert bool((dw == rows).all())


@pytest.mark.parametrize("rows", [0, 40, 9000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_status_of_a_weight_gradient(gc, dtype, rows):
    """Every field, whatever the workspace held."""
    ck, dy = gc.ActCheckpoint(rows, 72), torch.ones(rows, 40, device="cuda", dtype=dtype)
    gc.act_compress(torch.ones(rows, 72, device="cuda"), ck)
    ws = gc.act_weight_grad_workspace(rows, 40, 72, dtype)
    ws.fill_(0xA5)
    dw = torch.empty(40, 72, device="cuda")
    gc.act_weight_grad(dy, ck, dw, ws)
    d = gc.get_device_status(ws)
    assert (d.error_bits, d.exact_tensors, d.overflow_tensors, d.one_launch) == (0, 0, 0, 0)
    assert bool((dw == rows).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows, n, k", [(40, 8, 1), (40, 40, 7), (70, 130, 39), (500, 300, 254), (20, 24, 1459), (7000, 2600, 2598)])
def test_weight_grad_beside_other_columns(gc, rows, n, k, dtype):
    """Rows of dw on 16-byte boundaries that do not end on one: what lies between
    them is somebody else's, whatever the last columns hold."""
    x, dy = torch.ones(rows, k, device="cuda"), torch.ones(rows, n, device="cuda", dtype=dtype)
    ws = gc.act_weight_grad_workspace(rows, n, k, dtype)
    for spoiled in (False, True):
        ck, ld = gc.ActCheckpoint(rows, k), (k + 7) // 4 * 4
        if spoiled:
            x[rows // 2, k - 1] = float("nan")
        gc.act_compress(x, ck)
        for accumulate in (False, True):
            buf = torch.full((n, ld), 5.0, device="cuda")
            flat = buf.view(-1)
            # the last row ends with its columns, and with the matrix
            dw = flat[:(n - 1) * ld + k].as_strided((n, k), (ld, 1))
            gc.act_weight_grad(dy, ck, dw, ws, accumulate=accumulate)
            assert bool((buf[:, k:] == 5.0).all())
            last = (k - 1) // 32 * 32
            assert bool((dw[:, :last] == rows + 5.0 * accumulate).all())
            assert bool(torch.isnan(dw[:, last:]).all() if spoiled else (dw == rows + 5.0 * accumulate).all())
