"""What the sources of the step around the cache have to hold to, where a run
need not show it."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source(name):
    text = open(os.path.join(ROOT, "paged_kv_cache_41_gb300", "csrc", "kernels", name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_sums_are_changed_behind_a_barrier():
    # all[] is what every warp adds up; whoever writes it does so behind a barrier
    # that stands behind the last of those reads
    text = source("verify.cu")
    kernel = text[text.index("draft_verify_kernel(const VerifyArgs a)"):text.index("launch_draft_verify")]
    writes = [m.start() for m in re.finditer(r"\ball\[t\] -?= ", kernel)]
    reads = [m.end() for m in re.finditer(r"total \+= all\[s\]|part_of\(all\b|total_of\(row", kernel)]
    assert len(writes) == 2 and len(reads) == 6
    for at in writes:
        barrier = max(kernel.rfind("__syncthreads()", 0, at), kernel.rfind("cluster.sync()", 0, at))
        assert barrier > max([r for r in reads if r < at] + [0])
