"""Host-side checks of the norm + rotation kernel's source."""
import os
import re

from paged_kv_cache_slot_gb300 import build as bkv_build


def test_a_warps_reads_are_ordered_before_its_stores():
    """q_out may be q.  In the kernel of any shape a lane reads the element that turns with its own, which another lane
    stores: between the reads and the stores stands a barrier that orders memory (shuffles do not)."""
    with open(os.path.join(bkv_build.CSRC, "bkv_rope_write.cu")) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    src = src[src.index("rope_write_any_kernel(const Args a"):src.index("struct Piece")]
    last_read, store = src.rindex("src["), src.index("a.q_out")
    between = src[last_read:store]
    assert "__syncwarp();" in between
    # and it stands where every lane of the warp passes: outside of the loop over the elements
    before = src[src.index("float ss = 0.f;"):src.index("__syncwarp();", last_read)]
    assert before.count("{") == before.count("}")
