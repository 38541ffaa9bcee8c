"""The top of fp16's range in a checkpoint: what the header says reads back."""
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


def test_top_of_the_range(gc):
    x = torch.ones(3, 32, dtype=torch.float16)
    x[0, 0], x[0, 1] = 65248.0, -65024.0             # steps of 2^9: 127 of them
    x[1, 0], x[1, 1], x[1, 2] = 65280.0, 65024.0, -64992.0   # of 2^10: 63.75, 63.5 (to the even 64), 63.47
    x[2, 0] = 65504.0
    ck, half, wide = gc.ActCheckpoint(3, 32), torch.empty(3, 32, dtype=torch.float16, device="cuda"), torch.empty(3, 32, device="cuda")
    gc.act_compress(x.cuda(), ck)
    gc.act_decompress(ck, half)
    gc.act_decompress(ck, wide)
    inf = float("inf")
    assert half[0, :2].tolist() == [65024.0, -65024.0]
    assert half[1, :3].tolist() == [inf, inf, -64512.0] and half[2, 0] == inf
    assert wide[1, :3].tolist() == [65536.0, 65536.0, -64512.0] and wide[2, 0] == 65536.0
