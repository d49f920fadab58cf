"""Host-side checks of the draft verification kernel's source."""
import os
import re

from paged_kv_cache_slot_gb300 import build as bkv_build


def _kernel():
    with open(os.path.join(bkv_build.CSRC, "bkv_verify.cu")) as f:
        src = f.read()
    src = re.sub(r"//[^\n]*", "", src)
    return src[src.index("verify_kernel(const Args a)"):src.index("static int launch")]


def test_no_ctas_shared_memory_is_written_before_it_runs():
    """A CTA of a cluster may touch another's shared memory only once that CTA has started: every thread's arrival
    and wait at a cluster barrier come before the first mapped address."""
    src = _kernel()
    first = src.index("map_shared_rank")
    arrive, wait = src.find("barrier.cluster.arrive"), src.find("barrier.cluster.wait")
    assert 0 <= arrive < wait < first
    # neither stands in a branch: the body's own depth, behind its declarations
    for at in (arrive, wait):
        body = src[src.index("{"):at]
        assert body.count("{") - body.count("}") == 1
    # the loop's own barrier, once a pass, comes behind the write
    assert src.index("cluster.sync()") > first
