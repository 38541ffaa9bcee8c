"""Waits of the weight gradient's kernel, by its source: where all lanes of a
warp wait and go on to a vote or a barrier of the warp, they have to give up
together.  (A wait that runs out is not made on a GPU.)"""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_compression_gb300", "csrc",
                      "gc_wgrad.cu")


def test_whole_warps_give_up_together():
    with open(SOURCE) as f:
        text = f.read()
    unpack = text[text.index("if (warp < WG_CONV) {"):text.index("} else if (warp < WG_TMA) {")]
    write = text[text.index("bool wg_write("):text.index("template <int PARTS, bool TMA>\n__global__")]
    for role in (unpack, write):
        waits = re.findall(r"\bmbar_wait\w*", role)
        assert waits and set(waits) == {"mbar_wait_warp"}
        assert "_sync(FULL" in role or "__syncwarp" in role
    helper = re.search(r"bool mbar_wait_warp\(.*?\{(.*?)\}", text, re.S).group(1)
    assert "i < WG_POLLS" in helper and "if (__all_sync(FULL, mbar_poll(bar, parity))) return true;" in helper


def test_a_failed_call_sees_its_multiplications_end():
    """On a barrier that nothing else completes: an accumulator's own may be
    complete while the other one's chain is still being multiplied."""
    with open(SOURCE) as f:
        text = f.read()
    end = text[text.index("// MMAs in flight read this CTA's memory"):]
    commit, wait = re.search(r"mma_commit\((.*?)\);\s*mbar_wait\((.*), 0\);", end[:400]).groups() if "mbar_wait(drained, 0)" in end else ("", "")
    assert commit == wait == "drained"
    assert len(re.findall(r"\bdrained\b", text)) == 4           # its address, its setting up, and these two
    size = 8 * eval(re.search(r"bars\[(.*?)\]", text).group(1))
    assert int(re.search(r"drained = bar0 \+ (\d+)u", text).group(1)) + 8 <= size
