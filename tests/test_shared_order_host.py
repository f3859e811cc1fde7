"""Order of a copy behind the reads of the block it replaces, in the source of
the shared-prefix decode (no GPU): a copy out of order goes wrong too rarely
to be caught by its results alone."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "integer_only_quantized_b200", "csrc", "shared_kernel.cuh")


def _code():
    with open(SOURCE) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_own_blocks_are_replaced_behind_a_fence_and_a_barrier():
    code = _code()
    body = re.search(r"void issue\(const CUtensorMap\* tm[^{]*\{(.*?)\n  \}", code, re.S).group(1)
    order = [body.index(x) for x in ("fence_proxy_async_smem();", "__syncwarp();", "tma_load_3d_elect(")]
    assert order == sorted(order)
    # the ring's copies all go through it, and each that follows reads takes their value
    assert len(re.findall(r"tma_load_3d_elect\(", code)) == 1
    assert len(re.findall(r"read & a\.none", code)) == 2
