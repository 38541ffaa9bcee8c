"""The gradient norm's bits: set by sizes, types and places in a 16-byte granule."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
SIZES = [5, 4097, 100_003, 1, 333, 2_000_001]


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


def placed(values, dtype, granules, elements):
    """The values each in a buffer of its own, so many granules and elements from its start."""
    per, out = 16 // dtype.itemsize, []
    for i, v in enumerate(values):
        at = granules * (i % 3) * per + (elements + i) % per
        buf = torch.full((at + v.numel() + per,), 9.0, dtype=dtype, device="cuda")
        buf[at:at + v.numel()] = v
        out.append(buf[at:at + v.numel()])
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_same_offsets_same_bits(gc, dtype):
    gen = torch.Generator(device="cuda").manual_seed(31)
    values = [torch.randn(n, generator=gen, device="cuda").to(dtype) for n in SIZES]
    want = math.sqrt(math.fsum(float(v.double().square().sum()) for v in values))
    for elements in range(16 // dtype.itemsize):
        got = set()
        for granules in (0, 1, 7, 64):
            t, norm = placed(values, dtype, granules, elements), torch.empty(1, device="cuda")
            gc.grad_norm(t, norm, gc.grad_norm_workspace(t))
            got.add(float(norm))
        assert len(got) == 1
        assert abs(got.pop() - want) <= 18 * 2.0 ** -24 * want      # 32 squares and additions in fp32, then 64 bits
