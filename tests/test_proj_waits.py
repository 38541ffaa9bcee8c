"""Waits of the gated projection's kernel: by its source, and by a model of how a
pair of CTAs ends after one of them ran out.  (A wait that runs out is not made
on a GPU.)

What has to hold whichever wait gave up: no CTA of a cluster ends before the
copies and multiplications that reach its shared memory are done, and every
wait of the end is one that something in flight completes.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_compression_gb300", "csrc",
                      "gc_proj.cu")


@pytest.fixture(scope="module")
def kernel():
    with open(SOURCE) as f:
        text = f.read()
    begin = text.index("    k_gated_proj(const __grid_constant__ GpMaps maps")
    return text, text[begin:text.index("\n}\n", begin)]


def end_of(text):
    return re.search(r"void gp_drain\(.*?\n\}\n", text, re.S).group(0)


def test_whole_warps_give_up_together_and_in_time(kernel):
    text, body = kernel
    helper = re.search(r"bool gp_wait_warp\(.*?\{(.*?)\n\}\n", text, re.S).group(1)
    assert "i < GP_POLLS" in helper and "if (__all_sync(FULL, mbar_poll(bar, parity))) return true;" in helper
    # no other wait on a barrier, no time that stands for one
    assert len(re.findall(r"gp_wait_warp\(", body)) == 6 and len(re.findall(r"gp_wait_warp\(", end_of(text))) == 2
    assert not re.search(r"mbar_poll|mbar_wait|try_wait|test_wait|nanosleep|while \(true\)|for \(;;\)", body + end_of(text))


def test_a_wait_that_ran_out_is_told_to_the_whole_cluster(kernel):
    text, body = kernel
    tell = re.search(r"void gp_tell\(.*?\n\}\n", text, re.S).group(0)
    assert "c < ctas" in tell and "of_cta(smem_u32(lost), c)" in tell
    assert "const int ctas = (PAIR ? 2 : 1) * (joint ? a.splits : 1);" in body
    # the three roles, before they end
    join, end = body.index("  if (joint) {\n    // "), body.index("if (!ok) atomicOr(a.diag + DIAG_ERR, GC_DIAG_TIMEOUT);")
    cuts = [m.start() for m in re.finditer(r"// -+ (operands|MMA|result)\n", body)] + [join]
    assert len(cuts) == 4
    for role in (body[a:b] for a, b in zip(cuts, cuts[1:])):
        assert role.count("gp_tell(&lost, ctas);") == 1
        last = role[role.rindex("ok = gp_wait_warp("):]               # after its last wait, and wherever it gave up
        assert re.search(r"if \(!ok\) gp_tell\(&lost, ctas\);", last) or \
            (role.count("ok = ") == 1 and re.search(r"\) \{\s*gp_tell\(&lost, ctas\);\s*break;", last))
    # sums are only sent where all CTAs have theirs
    assert "cluster_sync();\n    const bool mine = warp >= GP_FIRST && quad < quads && lost == 0u;" in body[join:end]
    # what follows is gone through by all of them, whatever their own waits did
    after = body[end:]
    assert re.search(r"__syncthreads\(\);\n  if \(PAIR \|\| joint\) cluster_sync\(\);.*?\n  if \(lost != 0u\) \{", after)
    drain = after[after.index("if (lost != 0u) {"):]
    assert "ok" not in re.findall(r"\b\w+\b", re.sub(r"//.*", "", drain + end_of(text)))
    assert drain.index("gp_drain<BACK, PAIR, PARTS>(") < drain.index("__syncthreads();\n    if (PAIR || joint) cluster_sync();") < drain.index("dealloc")


def test_a_failed_call_sees_its_multiplications_end(kernel):
    """On a barrier that nothing else completes."""
    text, body = kernel
    drain = end_of(text)
    assert "gp_commit<PAIR>(bar0 + GP_DRAINED, leader)" in drain and "gp_wait_warp(bar0 + GP_DRAINED, 0u)" in drain
    assert len(re.findall(r"\bGP_DRAINED\b", text)) == 5           # its place and the next one's, its setting up, and these two
    assert "drained" not in body.replace("const uint32_t drained = bar0 + GP_DRAINED", "").replace("mbar_init(drained, 1)", "")
    assert drain.index("gp_commit<PAIR>(") < drain.index("gp_wait_warp(bar0 + GP_DRAINED, 0u)")
    assert not re.search(r"rank == 0[^;]*gp_wait_warp\(bar0 \+ GP_DRAINED", drain)              # both CTAs of a pair wait


# ------------------------------------------------------------------ the end of a pair, in a model

class Barrier:
    """An mbarrier of one arrival: complete when that came and no bytes are expected any more."""

    def __init__(self):
        self.phase, self.pending, self.bytes = 0, 1, 0

    def change(self, arrivals, expected):
        self.pending -= arrivals
        self.bytes += expected
        assert self.pending >= 0, "an arrival beyond the phase's"
        if self.pending == 0 and self.bytes == 0:
            self.phase, self.pending = self.phase + 1, 1

    def done(self, parity):
        return self.phase % 2 != parity


class Pair:
    """Stages of two CTAs: rank 0's copies and rank 1's land on rank 0's `full`, an
    MMA's end on both CTAs' `empty`.  Any wait whose phase is not complete may give up."""

    def __init__(self, rng, stages, slots):
        self.rng, self.stages, self.slots = rng, stages, slots
        self.full, self.empty = [Barrier() for _ in range(slots)], [[Barrier() for _ in range(slots)] for _ in range(2)]
        self.flying, self.multiplying, self.lost = [], [], False
        self.issued = [0, 0]

    def issue(self, rank):
        g = self.issued[rank]
        assert not any(f == (rank, g % self.slots) for f in self.flying), "a stage's room is still written"
        assert not any(m % self.slots == g % self.slots for m in self.multiplying), "a stage's room is still read"
        if rank == 0:
            self.full[g % self.slots].change(1, 2)
        self.flying.append((rank, g % self.slots))
        self.issued[rank] += 1

    def land(self):
        _, slot = self.flying.pop(self.rng.randrange(len(self.flying)))
        self.full[slot].change(0, -1)

    def multiplied(self):
        m = self.multiplying.pop(0)
        for rank in range(2):
            self.empty[rank][m % self.slots].change(1, 0)

    def producer(self, rank):
        for g in range(self.stages):
            if not (yield self.empty[rank][g % self.slots], (g // self.slots + 1) % 2):
                return
            self.issue(rank)
        for g in range(max(0, self.stages - self.slots), self.stages):
            if not (yield self.empty[rank][g % self.slots], g // self.slots % 2):
                return

    def product(self):
        for g in range(self.stages):
            if not (yield self.full[g % self.slots], g // self.slots % 2):
                return
            self.multiplying.append(g)

    def roles(self, patience):
        """Until all three have ended; gives up at random."""
        running = [(r, next(r)) for r in (self.producer(0), self.producer(1), self.product())]
        while running:
            r, (bar, parity) = running.pop(self.rng.randrange(len(running)))
            done = bar.done(parity)
            if done or self.rng.random() < patience:
                self.lost |= not done
                try:
                    running.append((r, r.send(done)))
                except StopIteration:
                    pass
            else:
                running.append((r, (bar, parity)))
            if self.flying and self.rng.random() < 0.3:
                self.land()
            if self.multiplying and self.rng.random() < 0.3:
                self.multiplied()

    def wait(self, bar, parity):
        while not bar.done(parity):
            assert self.flying, "a wait that nothing in flight completes"
            self.land()

    def end(self):
        """As the kernel does it."""
        if not self.lost:
            return
        while self.multiplying:
            self.multiplied()
        most = max(self.issued)
        for rank in range(2):
            while self.issued[rank] < most:
                self.issue(rank)
        for g in range(most - 1, max(0, most - self.slots) - 1, -1):
            self.wait(self.full[g % self.slots], g // self.slots % 2)

    def end_by_its_own_stages(self):
        """Each CTA waiting for its own count alone: the first one for its stages that can complete."""
        while self.multiplying:
            self.multiplied()
        n = min(self.issued)
        for g in range(max(0, n - self.slots), n):
            self.wait(self.full[g % self.slots], g // self.slots % 2)


def models():
    for seed in range(3000):
        rng = random.Random(seed)
        p = Pair(rng, rng.randrange(1, 40), rng.randrange(1, 9))
        p.roles(rng.choice((0.0, 0.002, 0.02, 0.2)))
        yield p


def test_a_pair_ends_with_nothing_in_flight():
    uneven = 0
    for p in models():
        uneven += p.issued[0] != p.issued[1]
        assert abs(p.issued[0] - p.issued[1]) <= p.slots
        p.end()
        assert not p.flying and not p.multiplying
    assert uneven > 100


def test_the_model_shows_what_was_left_in_flight():
    left = 0
    for p in models():
        p.end_by_its_own_stages()
        left += bool(p.flying)
    assert left > 0
