"""What the draft-tree kernel's source has to hold to, where a run could only
show it by hanging."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_each_warpgroup_moves_its_registers_by_one_instruction():
    # PTX: all threads of a warpgroup execute the same setmaxnreg.  Each share
    # of the registers belongs to one kind of warpgroup, so a share that is
    # named at two places is taken by warps of one group apart.
    path = os.path.join(ROOT, "paged_kv_cache_41_gb300", "csrc", "kernels", "draft_tc.cu")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    calls = re.findall(r"\b(give|take)_registers<(kDt\w+)>\(\)", text)
    assert sorted(calls) == [("give", "kDtMxIssueRegs"), ("give", "kDtMxWidenRegs"),
                             ("take", "kDtMxSoftRegs")]
    # and the branches above them part whole warpgroups, four warps each
    warps = {k: int(v) for k, v in re.findall(r"constexpr int (kDtSoftWarps|kDtWidenWarps) = (\d+);", text)}
    first = re.search(r"constexpr int kDtWidenFirst = kDtSoftWarps \+ (\d+);", text)
    assert warps["kDtSoftWarps"] % 4 == warps["kDtWidenWarps"] % 4 == int(first.group(1)) % 4 == 0
    before = text[:text.index("give_registers<kDtMxIssueRegs>()")]
    assert re.search(r"else if \(warp >= kDtSoftWarps && warp < kDtWidenFirst\) \{\s*if \(kMx\)\s*$", before)


def test_a_failed_query_is_not_kept():
    # the launcher may keep what the attribute query said, not that it failed:
    # no initialiser of a static holds the query
    path = os.path.join(ROOT, "paged_kv_cache_41_gb300", "csrc", "kernels", "draft_tc.cu")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    assert "cudaFuncGetAttributes" in text
    for m in re.finditer(r"static [^;]*?=\s*\[&\]\s*\{.*?\}\(\);", text, flags=re.S):
        assert "cudaFuncGetAttributes" not in m.group(0)
