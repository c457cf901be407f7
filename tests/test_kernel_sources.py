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


def kernels(text):
    """(signature, body) of every __global__ function of a source."""
    for m in re.finditer(r"__global__", text):
        head = text.index("{", m.start())
        depth, at = 1, head + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield text[m.start():head], text[head:at]


@pytest.mark.parametrize("name", ["k_ortho.cu", "k_combine_norm.cu"])
def test_what_the_kernel_before_writes_is_not_read_as_constant(name):
    """A kernel that begins while the one before it still writes waits for that one's end (griddepcontrol.wait) and then
    reads what it left.  The read-only path (__ldg, or const __restrict__, which the compiler may read by it) is
    defined for data that nobody writes during the kernel."""
    constant = {"column_sums_kernel": {"w_post", "res_scale"}}  # what the caller gave
    seen = 0
    for head, body in kernels(source(name)):
        if "griddepcontrol.wait" not in body:
            continue
        seen += 1
        kernel = re.search(r"(\w+)\s*\($", head[:head.rindex("(") + 1]) or re.search(r"(\w+_kernel)", head)
        allowed = constant.get(kernel.group(1), set())
        read_only = set(re.findall(r"const \w+\s*\*\s*__restrict__ (\w+)", head)) - allowed
        assert not read_only, (kernel.group(1), read_only)
        assert "__ldg(" not in body, kernel.group(1)
    assert seen
