"""Rules of the kernels' sources that no run can check: the cases that they are for must not come up on a GPU.  CPU only."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "token_dispatch_gb300", "csrc")


def source(name):
    """A source without its comments, on one line."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", f.read()))


@pytest.mark.parametrize("name", ["k_ortho.cu", "k_w4.cu", "k_gemm_tc.cu"])
def test_warps_agree_on_the_end_of_a_wait_for_sums(name):
    """A bounded wait that gives up may end differently in the lanes of a warp.  What follows a wait for sums in tensor
    memory (tcgen05.ld, __syncwarp) is for the whole warp: it asks all lanes before it goes on or leaves."""
    text = source(name)
    waits = [m.start() for m in re.finditer(r"wait_(?:bounded|lazily)\((?:accf|dw_bar)", text)]
    assert waits
    for at in waits:
        assert text[:at].endswith("__all_sync(0xffffffffu, "), text[at - 60:at + 60]


@pytest.mark.parametrize("name", ["k_ortho.cu", "k_w4.cu", "k_gemm_tc.cu"])
def test_products_under_way_are_waited_for_before_tensor_memory_is_given_back(name):
    """A kernel that gave up on a wait may still have products under way: it waits for them, with a limit of its own,
    before it frees the tensor memory that they write."""
    text = source(name)
    spans = re.findall(r"tcgen05\.alloc.*?tcgen05\.dealloc", text)
    assert spans and len(spans) == text.count("tcgen05.alloc")
    for span in spans:
        assert "DRAIN_LIMIT" in span, span[:80]
