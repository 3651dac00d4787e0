"""What the memory model asks of the few-token kernels' source and no run can show (no GPU needed)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tp_reduce_moe_gb300", "csrc")


def body(name, text):
    """The text of a function's body, from its first brace to the one that closes it."""
    start = text.index("{", text.index(name))
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(name)


def test_masks_in_the_ring_are_fenced_before_the_copies():
    """The expert masks lie where the first copies land: behind every thread's last access a proxy fence, then the barrier."""
    text = open(os.path.join(CSRC, "moe_experts.cu")).read()
    build = re.sub(r"//[^\n]*", "", body("void build_items", text))
    tail = build[build.rindex("mask["):]
    assert "fence_proxy_async();" in tail
    assert tail.index("fence_proxy_async();") < tail.rindex("__syncthreads();")
    common = open(os.path.join(CSRC, "moe_common.cuh")).read()
    assert "fence.proxy.async.shared::cta" in body("void fence_proxy_async", common)
