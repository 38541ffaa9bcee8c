"""How the gated projection cuts calls, without a GPU: every cut is one that the
kernel can take, and the sizes that the GPU tests run take all of them."""
import ctypes as C

import pytest

import _proj_cuts as cuts

RING, M, K, SLOTS = 192 * 1024, 128, 64, 12


@pytest.fixture(scope="module")
def lib():
    return cuts.library()


@pytest.fixture(scope="module")
def gc():
    from gradient_compression_gb300 import build
    build.build()
    import gradient_compression_gb300 as gcmod
    return gcmod


EXTREME = [(1, 1, 1), (1, 1, 2 ** 31 - 1), (129, 1, 2 ** 24), (2 ** 31 - 1, 1, 1), (2 ** 20, 32, 16), (128, 2 ** 22, 1), (127, 16, 2 ** 22),
           (1, 2 ** 31 - 1, 1), (257, 31, 2 ** 20), (16384, 14336, 8192)]


@pytest.mark.parametrize("held", [cuts.HELD, (152, 70, 40, 30, 20, 15, 10, 8), (0,) * 8], ids=["whole", "fewer", "none"])
@pytest.mark.parametrize("mode", cuts.MODES)
def test_every_cut_is_possible(lib, gc, mode, held):
    back = mode == "back"
    sizes = cuts.draws(3, 5000) + EXTREME
    size = C.c_size_t(0)
    for (rows, n, k), plan in zip(sizes, cuts.plans(lib, mode, sizes, held)):
        pair, apart, bn, parts, tm, tn, splits, span = plan
        cols, summed = (k, n) if back else (n, k)
        blocks = -(-summed // K)
        steps = (2 if back else 1) * -(-blocks // parts)
        assert (tm - 1) * M * (1 + pair) < rows <= tm * M * (1 + pair) and (tn - 1) * bn < cols <= tn * bn
        assert not (pair and rows <= M)
        # an MMA's columns, and both accumulators in tensor memory
        wide = bn if back else 2 * bn
        assert 32 <= wide <= 256 and wide % 16 == 0 and (bn % 32 == 0 or mode == "out")
        # the ring holds two stages at least
        stage = parts * lib.proj_stage(rows, bn, pair, int(back))
        assert 2 * stage <= RING and min(SLOTS, RING // stage) >= 2
        # all of the sum, none of it twice, no split without any
        assert (splits - 1) * span < steps <= splits * span
        if splits > 1:
            assert tm * tn * splits <= (cuts.SMS // 2 if pair else cuts.SMS)
        if apart:
            assert back and gc.lib().gc_gated_proj_backward_workspace_size(rows, n, k, 0, C.byref(size)) == gc.GC_OK
            assert size.value >= 4 * splits * rows * (-(-k // 8) * 8) + 16
        elif splits > 1:
            assert splits * (1 + pair) <= 8 and tm * tn <= held[splits * (1 + pair) - 1]
            assert lib.proj_fits(-(-bn // 32), splits, int(back))


@pytest.mark.parametrize("mode", cuts.MODES)
def test_the_sizes_run_on_the_gpu_take_every_cut(lib, mode):
    """Of other draws of the same range at most one in a thousand is cut in another way."""
    run = set(cuts.cases(lib, mode))
    assert {what[0] for what in run} >= {0, 1} and (mode != "out" or {("few", 1), ("few", 2), ("few", 3)} <= run)
    widths = range(32, 129, 16) if mode == "out" else range(32, 129 if mode == "held" else 257, 32)
    assert {(w[0], w[1]) for w in run if w[0] != "few"} == {(pair, bn) for pair in (0, 1) for bn in widths}
    other = cuts.kinds(lib, mode, cuts.draws(8, 20000))
    assert sum(len(sizes) for what, sizes in other.items() if what not in run) <= 20
