"""The mx4 expert products' kernels one by one: many tiles in a row through each pair kernel."""
import pytest
import torch

import mx4_plain as mp
import top_routing_grouped_noisy_b200 as moe
from test_gpu_mx4 import _Routed

pytestmark = pytest.mark.gpu


def _batch(T, E, m, d, k=2):
    """A routed batch with random experts, h of its first product made."""
    g = torch.Generator(device="cuda").manual_seed(T + m)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].cpu()
    W = moe.Mx4Experts.quantize(r(E, 2 * mp.up(m, 16), d), r(E, d, mp.up(m, 8)), E, m, d)
    rt = _Routed(idx, r(T, d), E, m)
    up = lambda: moe.moe_expert_up_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, W, rt.h_q, rt.h_s, rt.ws)
    down = lambda: moe.moe_expert_down_mx4(rt.p, rt.h_q, rt.h_s, rt.offsets, W, rt.out, rt.ws)
    return rt, up, down


@pytest.mark.parametrize("m", [688, 1600])
def test_many_tiles_in_a_row(m):
    """Each pair takes several tiles through both accumulators, A resident (m = 688) and
    streamed; beside copies that slow the epilogue's stores now and then, the bits stay."""
    rt, up, down = _batch(8192, 4, m, 1024)
    up()
    down()
    torch.cuda.synchronize()
    ref = rt.h_q.clone(), rt.h_s.clone(), rt.out.clone()
    a = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    b, side = torch.empty_like(a), torch.cuda.Stream()
    for i in range(24):
        rt.h_q.fill_(0x55)
        rt.out.fill_(7.0)
        if i % 3:
            with torch.cuda.stream(side):
                b.copy_(a)
        up()
        down()
        assert torch.equal(rt.h_q, ref[0]) and torch.equal(rt.h_s, ref[1])
        assert torch.equal(rt.out, ref[2])
    side.synchronize()
    assert moe.moe_get_device_status(rt.ws) == 0


LIMIT_NS = 2_000_000_000


def _runs_out(ws, call, tries=3000):
    """Whether `call`, with a wait limit of 0 and nothing in L2, reports a wait that ran out.
    mbarrier.try_wait suspends the thread for some microseconds of its own and a limit is first
    compared after two of them, so that most waits of a product are over before: of 40 calls, 1
    to 40 report one, by size.  Calls are repeated until one does."""
    for _ in range(tries):
        torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        moe.moe_set_wait_limit_ns(0)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            moe.moe_set_wait_limit_ns(LIMIT_NS)
        status = moe.moe_get_device_status(ws)
        assert status in (0, moe.MOE_ERR_DEVICE_TIMEOUT)
        if status != 0:
            return True
    return False


# one CTA a tile; pairs, A resident in the second product (m <= 1536); pairs, A streamed
@pytest.mark.parametrize("T,E,m,d", [(250, 16, 4096, 4096), (16000, 4, 1376, 4096),
                                     (4000, 2, 4096, 4096)])
def test_each_product_reports_its_wait(T, E, m, d):
    """Each product of its own reports MOE_ERR_DEVICE_TIMEOUT when its waits run out, returns, and
    is right in the next call."""
    rt, up, down = _batch(T, E, m, d)
    up()
    down()
    ref = rt.h_q.clone(), rt.out.clone()
    assert moe.moe_get_device_status(rt.ws) == 0
    for call, buf, want in ((up, rt.h_q, ref[0]), (down, rt.out, ref[1])):
        assert _runs_out(rt.ws, call)
        buf.zero_()
        call()
        assert torch.equal(buf, want) and moe.moe_get_device_status(rt.ws) == 0


def test_few_token_barrier_reports_its_wait():
    """The same for the grid barrier of the few-token layer: with one expert of 16 neurons all
    CTAs but one wait there from the start.  The barrier's count serves the next launch."""
    from test_gpu_mx4 import _Layer
    L = _Layer(T=1, E=1, k=1, m=16, d=32)
    ref = L.run(moe.MX4_ACT_BF16).y.clone()
    for _ in range(3):
        assert _runs_out(L.ws, lambda: L.run(moe.MX4_ACT_BF16))
        for _ in range(3):
            assert torch.equal(L.run(moe.MX4_ACT_BF16).y, ref)
        assert moe.moe_get_device_status(L.ws) == 0
