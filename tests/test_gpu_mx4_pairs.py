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
