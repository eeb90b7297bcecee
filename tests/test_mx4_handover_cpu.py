"""How the mx4 pair kernels hand accumulator columns back to the issuer, read from the source: a
tcgen05.ld is ordered before an arrival on an mbarrier only by tcgen05.fence::before_thread_sync,
so the arrival may not stand anywhere without it."""
import os
import re

import top_routing_grouped_noisy_b200 as moe

SRC = os.path.join(os.path.dirname(moe.__file__), "csrc", "mx4_gemm.cu")


def _body(text, head):
    """The braces that follow `head`."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError("no end of " + head)


def test_every_arrival_follows_the_fence():
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    hand_over = _body(text, "void hand_over(")
    order = [hand_over.index(s) for s in ("tc_fence_before()", "__syncwarp()", "mbar_arrive_cluster(")]
    assert order == sorted(order)
    # the definition and the one use
    assert len(re.findall(r"\bmbar_arrive_cluster\(", text)) == 2
    # both halves of both pair kernels' epilogues
    assert len(re.findall(r"\bhand_over\(tfree0", text)) == 4
    # the kernel of single CTAs: fence, whole warp, arrival
    one = _body(text, "mx4_gemm_kernel(")
    at = one.index("mbar_arrive(smem_u32(&aux->tempty")
    before = one[:at]
    assert before.rindex("tmem_wait_ld()") < before.rindex("tc_fence_before()") < \
        before.rindex("__syncwarp()")
