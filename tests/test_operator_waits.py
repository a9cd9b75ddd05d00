"""The waits of the 4-bit product's kernel, as its source has them (a wait that
runs out cannot be tried on a GPU that works)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kernel():
    text = open(os.path.join(ROOT, "hash_table_cache_gb300", "csrc", "mx_matmul.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    start = text.index("matmul_kernel(const __grid_constant__ Maps maps")
    return text[start:text.index("__global__ void zero_kernel")]


def test_roles_of_whole_warps_wait_as_warps(kernel):
    """The warps that read the accumulators run tcgen05.ld.sync.aligned after
    their wait: all lanes of a warp have to leave it with one answer.  The other
    roles are one elected thread."""
    loading, rest = kernel.split("warp == 0 && elect()")[1].split("warp == 1 && half_of == 0 && elect()")
    issuing, reading = rest.split("else if (warp >= 2)")
    for role in (loading, issuing):
        assert re.search(r"\bwait\(", role) and "wait_warp" not in role and "sync.aligned" not in role
    assert "wait_warp(" in reading and not re.search(r"\bwait\(", reading)


def test_a_warp_wait_is_a_vote():
    text = open(os.path.join(ROOT, "hash_table_cache_gb300", "csrc", "mx_matmul.cu")).read()
    body = re.search(r"bool wait_warp\(uint64_t\* bar, uint32_t parity\) \{(.*?)\}", text, re.S).group(1)
    assert "__all_sync(0xFFFFFFFFu, wait(bar, parity))" in body


def test_a_block_ends_after_its_loads(kernel):
    """Where the issuing thread gives up, on either of its waits, it waits for the
    loads that follow in the order of the stages before it ends: the loading
    thread may have issued its last load and be gone."""
    issuing = kernel.split("warp == 1 && half_of == 0 && elect()")[1].split("else if (warp >= 2)")[0]
    for name in ("drained[b]", "full[s]"):
        assert re.search(r"if \([^;{]*!wait\(&" + re.escape(name) + r"[^{;]*\{\s*ok = false;\s*break;", issuing), name
    given_up = issuing[issuing.rindex("if (!ok) {"):]
    assert re.search(r"for \(int i = 0; i < S::kStages && wait\(&full\[s\], parity\); \+\+i\)\s*"
                     r"if \(\+\+s == S::kStages\) \{\s*s = 0;\s*parity \^= 1;", given_up)
