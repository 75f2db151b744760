"""The order of the two writers of a CTA's part records, read from the kernels' sources.

Every call clears both records of every CTA (lanes 0 and 1 of a warp), and a part of a cut
unit writes its record later, from another thread.  The second write has to happen after the
first: the clearing lanes and the thread that lets the others go on need a warp or block
barrier between them, as an arrival by lane 0 alone orders nothing that lane 1 wrote, and
shuffles and votes order no memory at all.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_gqa_flash_attention_gb300", "csrc")
CLEAR = re.compile(r"if \((?:lane|tid) < 2\) a\.part_info\[[^;]*\] = make_int4\(0, 0, 0, 0\);")


def between(name, to):
    """The source of `name` from behind the clearing to the first `to` behind it, without comments."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    found = list(CLEAR.finditer(src))
    assert len(found) == 1
    rest = src[found[0].end():]
    assert to in rest
    return rest[:rest.index(to)]


def test_the_tile_kernel_orders_its_cleared_records_before_the_parts_are_published():
    code = between("paged_tiles.cu", "mbar_arrive(smem_u32(&bar_seg_full")
    assert "__syncwarp();" in code


@pytest.mark.parametrize("name", ["paged_short.cu", "paged_f32.cu"])
def test_the_other_kernels_have_a_block_barrier_there(name):
    assert "__syncthreads();" in between(name, "paged_record(g)")
