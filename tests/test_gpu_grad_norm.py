"""Global gradient norm and clipping against plain 64-bit forms.

Tolerances.  Squares are summed in fp32 over at most 32 elements: each square and
each of at most 32 additions rounds by 2^-24, so a sum is within 33 2^-24 of its
value, its root within half of that; beyond, sums are in 64 bits; the norm itself is rounded
once: 17.5 2^-24 in all, 18 2^-24 with the 64-bit sums' own errors.  Clipped
values are the roundings of c * g in fp32, and of that to the type, with c the
rounded quotient: exact from the norm that was returned.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = 18 * 2.0 ** -24


@pytest.fixture(scope="module")
def gc(cuda_device):
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


def norm_of(gc, tensors, ws=None):
    norm = torch.full((3,), 7.0, device="cuda")
    gc.grad_norm(tensors, norm[1:2], gc.grad_norm_workspace(tensors, "cuda") if ws is None else ws)
    assert float(norm[0]) == float(norm[2]) == 7.0
    return float(norm[1])


def norm64(tensors):
    return math.sqrt(math.fsum(float((t.double().cpu() ** 2).sum()) for t in tensors))


def some(sizes, types, gen, off=0):
    """Tensors of these sizes at any element of their buffers, scales of their own."""
    out = []
    for i, n in enumerate(sizes):
        dt = DT[types[i % len(types)]]
        buf = (10.0 ** float(torch.rand((), generator=gen) * 4 - 3) * torch.randn(n + 9, generator=gen)).to(dt).cuda()
        o = (off + i) % 9
        out.append(buf[o:o + n])
    return out


LISTS = [[1], [0, 5, 0], [3, 31, 32, 33, 255, 256, 257], [4095, 4096, 4097, 1, 8191, 8192, 8193], [100_003], [1 << 20, 7, 999_999],
         [5] * 17, list(range(200)), [64] * 1500, [3_000_000, 1] + [1000] * 1100]


@pytest.mark.parametrize("types", [["f32"], ["bf16"], ["f16"], ["f32", "bf16", "f16"]])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}of{sum(s)}")
def test_norm_and_clip(gc, sizes, types):
    gen = torch.Generator().manual_seed(len(sizes) + sum(sizes))
    tensors = some(sizes, types, gen)
    want = norm64(tensors)
    got = norm_of(gc, tensors)
    assert abs(got - want) <= REL * want
    assert norm_of(gc, tensors) == got
    norm = torch.tensor([got], device="cuda")
    before = [t.clone() for t in tensors]
    # into an arena, in fp32 and in other types; clipped and not
    for most in (0.25 * got, 2.0 * got, math.inf, 0.0):
        c = np.float32(most) / np.float32(got) if got > np.float32(most) else np.float32(1)
        for out_type in ("f32", "bf16", "f16"):
            for gap in (0, 1):
                arena = torch.full((sum(sizes) + gap * (len(sizes) + 1),), 77.0, dtype=DT[out_type], device="cuda")
                views, at = [], gap
                for n in sizes:
                    views.append(arena[at:at + n])
                    at += n + gap
                gc.grad_clip(tensors, norm, most, out=views)
                flat = torch.cat([t.float() for t in tensors]) if sum(sizes) else torch.empty(0, device="cuda")
                ref = (flat * float(c)).to(DT[out_type])
                assert torch.equal(torch.cat([v for v in views]), ref)
                if gap:
                    keep = torch.ones_like(arena, dtype=torch.bool)
                    at = gap
                    for n in sizes:
                        keep[at:at + n] = False
                        at += n + gap
                    assert bool((arena[keep] == 77.0).all())
    assert all(torch.equal(t, b) for t, b in zip(tensors, before))
    # in place
    gc.grad_clip(tensors, norm, 2.0 * got)
    assert all(torch.equal(t, b) for t, b in zip(tensors, before))
    c = np.float32(0.25 * got) / np.float32(got)
    gc.grad_clip(tensors, norm, 0.25 * got)
    assert all(torch.equal(t, (b.float() * float(c)).to(b.dtype)) for t, b in zip(tensors, before))


@pytest.mark.parametrize("dtype", list(DT))
def test_range(gc, dtype):
    """Squares past fp32's range, above and below, beside ordinary ones."""
    dt = DT[dtype]
    top, low = float(torch.finfo(dt).max), float(torch.finfo(dt).smallest_normal)
    gen = torch.Generator().manual_seed(1)
    base = torch.randn(5000, generator=gen)
    for scale in (low * 2.0 ** -6, low * 8, 1e-4, 1.0, top / 64, top / 8):
        t = [(base * scale).to(dt).cuda(), torch.zeros(3000, dtype=dt, device="cuda"), (base[:777] * scale).to(dt).cuda()]
        want = norm64(t)
        got = norm_of(gc, t)
        if want <= 3.4e38:
            assert abs(got - want) <= REL * want + 2.0 ** -150, (scale, got, want)
        else:
            assert got == math.inf
    mixed = torch.zeros(10_000, dtype=dt)
    mixed[17], mixed[18], mixed[9000] = low, 1.0, low
    assert abs(norm_of(gc, [mixed.cuda()]) - norm64([mixed])) <= REL
    assert norm_of(gc, [torch.zeros(100_000, dtype=dt, device="cuda")]) == 0.0
    assert norm_of(gc, []) == 0.0 and norm_of(gc, [torch.empty(0, dtype=dt, device="cuda")]) == 0.0
    one = torch.zeros(70_000, dtype=dt)
    for at in (0, 1, 8, 4095, 69_999):
        x = one.clone()
        x[at] = -3.0
        assert norm_of(gc, [x.cuda()]) == 3.0


@pytest.mark.parametrize("dtype", list(DT))
def test_not_finite(gc, dtype):
    dt = DT[dtype]
    x = torch.ones(9001, dtype=dt)
    for bad, want in ((math.inf, math.inf), (-math.inf, math.inf), (math.nan, math.nan)):
        for at in (0, 5, 4096, 9000):
            y = x.clone()
            y[at] = bad
            t = [x.cuda(), y.cuda()]
            got = norm_of(gc, t)
            assert got == want or (math.isnan(got) and math.isnan(want))
            norm = torch.tensor([got], device="cuda")
            out = [torch.empty(9001, device="cuda") for _ in range(2)]
            gc.grad_clip(t, norm, 1.0, out=out)
            if math.isnan(want):                 # as they are
                assert torch.equal(out[0], t[0].float()) and torch.equal(out[1].nan_to_num(5.0), t[1].float().nan_to_num(5.0))
            else:                                # times 1 / infinity
                assert bool((out[0] == 0).all()) and bool(torch.isnan(out[1][at])) and int(torch.isnan(out[1]).sum()) == 1


def test_any_order_of_dimensions(gc):
    gen = torch.Generator().manual_seed(2)
    base = torch.randn(6, 10, 14, 3, generator=gen).cuda()
    views = [base.permute(0, 3, 1, 2), base[0].t() if base.dim() == 2 else base[1].permute(2, 0, 1), torch.randn((), generator=gen).cuda()]
    assert abs(norm_of(gc, views) - norm64(views)) <= REL * norm64(views)
    outs = [torch.empty_like(v) for v in views]
    norm = torch.tensor([2.0], device="cuda")
    gc.grad_clip(views[:1] + views[2:], norm, 1.0, out=outs[:1] + outs[2:])
    assert torch.equal(outs[0], views[0] * 0.5) and torch.equal(outs[2], views[2] * 0.5)
    flat = torch.empty(base.numel(), device="cuda")
    gc.grad_clip([base], norm, 1.0, out=[flat])
    assert torch.equal(flat, base.reshape(-1) * 0.5)
    for tensors, out in (([base[:, ::2]], None), ([base[..., :1].expand(6, 10, 14, 3)], None), ([views[0]], [torch.empty(6, 3, 10, 14, device="cuda")]),
                         ([base], [base[:1]]), ([base], []), ([base.int()], None), ([base.to_sparse()], None)):
        with pytest.raises(ValueError):
            gc.grad_clip(tensors, norm, 1.0, out=out)
    with pytest.raises(gc.GCError):
        gc.grad_clip([base, base], norm, 1.0)
    with pytest.raises(gc.GCError):
        gc.grad_clip([base], norm, -1.0)
    with pytest.raises(ValueError):
        gc.grad_norm([base], torch.empty(2, device="cuda"), gc.grad_norm_workspace([base]))
    with pytest.raises(gc.GCError):
        gc.grad_norm([base], norm, gc.grad_norm_workspace([base])[:100])


def test_streams_and_graphs(gc):
    gen = torch.Generator().manual_seed(3)
    tensors = some([1000, 4097, 300_000, 3], ["f32", "bf16"], gen)
    ws, norm = gc.grad_norm_workspace(tensors), torch.empty(1, device="cuda")
    out = [torch.empty(t.numel(), device="cuda") for t in tensors]

    def step(stream=None):
        gc.grad_norm(tensors, norm, ws, stream=stream)
        gc.grad_clip(tensors, norm, 0.5, out=out, stream=stream)

    step()
    want = [float(norm)] + [o.clone() for o in out]
    for o in out:
        o.zero_()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    step(other)
    other.synchronize()
    assert float(norm) == want[0] and all(torch.equal(o, w) for o, w in zip(out, want[1:]))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for factor in (2.0, 0.25):
        for t in tensors:
            t.mul_(factor)
        graph.replay()
        got = [norm.clone()] + [o.clone() for o in out]
        step()
        assert torch.equal(got[0], norm) and all(torch.equal(a, b) for a, b in zip(got[1:], out))


def test_long(gc):
    """A tensor of more than 2^31 elements."""
    n = (1 << 31) + 12_345
    t = torch.zeros(n, dtype=torch.float16, device="cuda")
    for at in (0, (1 << 31) - 1, 1 << 31, n - 1):
        t[at] = 2.0
    assert norm_of(gc, [t]) == 4.0
    out = torch.ones(n, dtype=torch.float16, device="cuda")
    gc.grad_clip([t], torch.tensor([4.0], device="cuda"), 2.0, out=[out])
    assert float(out[(1 << 31):].float().sum()) == 2.0 and float(out[:4096].float().sum()) == 1.0
    t.mul_(0.5)
    assert torch.equal(out, t)


def test_a_step_before_compression(gc):
    """Gradients of several types, clipped into the arena, then Top-k: the same as of the arena clipped by hand."""
    gen = torch.Generator().manual_seed(11)
    sizes = [5000, 33, 70_000, 1024]
    grads = some(sizes, ["bf16", "f32"], gen)
    off = np.concatenate(([0], np.cumsum(sizes)))
    layout = gc.Layout(off, [50, 1, 700, 10], device="cuda")
    arena = torch.empty(int(off[-1]), device="cuda")
    norm = torch.empty(1, device="cuda")
    gc.grad_norm(grads, norm, gc.grad_norm_workspace(grads))
    gc.grad_clip(grads, norm, 0.5, out=list(arena.split(sizes)))
    by_hand = torch.cat([g.float() for g in grads]) * (np.float32(0.5) / np.float32(float(norm))).item()
    assert torch.equal(arena, by_hand)
    comp = gc.TopkCompressor(layout, gc.GC_EF)
    e = torch.zeros_like(arena)
    idx, val, _, _ = comp(arena, e, seed=1, it=0)
    got = idx.clone(), val.clone()
    e.zero_()
    idx, val, _, _ = comp(by_hand, e, seed=1, it=0)
    assert torch.equal(got[0], idx) and torch.equal(got[1], val)


def test_some_in_place_and_some_not(gc):
    gen = torch.Generator().manual_seed(21)
    tensors = some([5000, 77, 300, 9001], ["f32", "bf16"], gen)
    before = [t.clone() for t in tensors]
    outs = [tensors[0], torch.empty(77, device="cuda"), tensors[2], torch.empty(9001, dtype=torch.float16, device="cuda")]
    norm = torch.tensor([8.0], device="cuda")
    for most in (4.0, 16.0):
        for t, b in zip(tensors, before):
            t.copy_(b)
        gc.grad_clip(tensors, norm, most, out=outs)
        for o, b in zip(outs, before):
            assert torch.equal(o, (b.float() * min(1.0, most / 8.0)).to(o.dtype))
        assert torch.equal(tensors[1], before[1]) and torch.equal(tensors[3], before[3])
    with pytest.raises(gc.GCError):                    # an output that is another one's input
        gc.grad_clip(tensors, norm, 4.0, out=[tensors[0], tensors[2][:77], tensors[2], outs[3]])


def test_two_norms_at_once(gc):
    """On two streams, each with a workspace of its own; then one workspace by call after call."""
    gen = torch.Generator().manual_seed(22)
    lists = [some([300_000, 5, 70_000], ["f32"], gen), some([100_000] * 20, ["bf16"], gen)]
    want = [norm_of(gc, t) for t in lists]
    norms, spaces = [torch.zeros(1, device="cuda") for _ in lists], [gc.grad_norm_workspace(t) for t in lists]
    streams = [torch.cuda.Stream() for _ in lists]
    torch.cuda.synchronize()
    for _ in range(10):
        for t, n, w, s in zip(lists, norms, spaces, streams):
            gc.grad_norm(t, n, w, stream=s)
    torch.cuda.synchronize()
    assert [float(n) for n in norms] == want
    ws = gc.grad_norm_workspace(lists[1])
    for t, n in zip(lists + lists[::-1], want + want[::-1]):
        assert norm_of(gc, t, ws) == n
