"""The end of the gated projection's CTAs after a wait that ran out, by the
kernel's own code on the host: from wherever either CTA of a pair gave up, the
one that is behind issues exactly the other one's further stages, and the first
one waits for every stage that may be in flight, by the parity of its turn."""
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gradient_compression_gb300", "csrc")


def extracted():
    """The types, the order of items and the two functions, without what only a GPU has."""
    with open(os.path.join(CSRC, "gc_proj.cu")) as f:
        text = f.read()

    def part(begin, end):
        at = text.index(begin)
        return text[at:text.index(end, at) + len(end)]

    parts = [re.search(r"constexpr int GP_SLOTS = \d+;", text).group(0), part("struct GpMaps {", "\n};"), part("struct GpArgs {", "\n};"),
             part("struct GpItem {", "\n};"), part("__device__ __forceinline__ GpItem gp_item(", "\n}"), part("struct alignas(8) GpFed {", "\n};"),
             part("constexpr uint32_t GP_EMPTY", ";\n"), part("template <bool BACK, bool PAIR, int PARTS>\n__device__ __forceinline__ void gp_feed(", "\n}"),
             part("template <bool BACK, bool PAIR, int PARTS>\n__device__ __noinline__ void gp_drain(", "\n}")]
    code = re.sub(r"__device__ __(forceinline|noinline)__", "static", "\n".join(parts))
    code, found = re.subn(r'asm volatile\("ld\.shared::cluster\.v2\.u32 \{%0, %1\}, \[%2\];" : "=r"\(i\), "=r"\(s\) : "r"\(there\) : "memory"\);',
                          "check_there(there), i = there_i, s = there_s;", code)
    assert found == 1 and "asm" not in code
    return "static void check_there(uint32_t at) { if (at >> 28 != (blockIdx.x & 1u ^ 1u)) std::abort(); }\n" + code


def test_a_pair_ends_from_every_place(tmp_path):
    (tmp_path / "extracted.h").write_text(extracted())
    exe = str(tmp_path / "drain")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-I", str(tmp_path), "-I", CSRC,
                    os.path.join(HERE, "_proj_drain.cpp"), "-o", exe], check=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout == "done\n", p.stdout
