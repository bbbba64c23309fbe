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


def test_a_decode_of_empty_sequences_waits_too():
    # a kernel that is launched early has to wait for the one in front of it, or it
    # may be over, and the next one begin, before that is: CTAs without work may
    # leave, but not all of them
    leave = re.search(r"if \(lo >= hi\)(.*?)return 0;", source("plan.cuh"), flags=re.S).group(1)
    assert "if (S == 0) pdl_wait();" in leave
    # and in the split without a plan the first CTA of each sequence, which has its
    # result to write
    for name in ("window_mma.cu", "decode_partial.cuh"):
        text = source(name)
        assert re.search(r"if \(n < 0\) \{\s*if \(a\.plan_before_wait\) pdl_wait\(\);", text[:text.index("if (n <= 0)")])
