"""The mx4 handles on the GPU: tensors whose storage is replaced between calls, and copies."""
import copy
import pickle

import pytest
import torch

import top_routing_grouped_noisy_b200 as moe
from test_gpu_mx4 import _Layer

pytestmark = pytest.mark.gpu
ACTS = [moe.MX4_ACT_BF16, moe.MX4_ACT_MX4]
WEIGHTS = ("W13_q", "W13_s", "W2_q", "W2_s")


def _pair():
    """Two layers of one shape, other weights, the same inputs."""
    A, B = (_Layer(T=7, E=4, k=2, m=96, d=256, seed=s) for s in (1, 2))
    B.dev = A.dev
    return A, B


@pytest.mark.parametrize("act", ACTS)
def test_weights_swapped_in_place(act):
    """The calls multiply with the weights that the handle's tensors hold at that moment."""
    A, B = _pair()
    ya, yb = A.run(act).y.clone(), B.run(act).y.clone()
    assert not torch.equal(ya, yb)
    kept = [(getattr(A.W, n).data, getattr(B.W, n).data) for n in WEIGHTS]
    for n, (_, new) in zip(WEIGHTS, kept):
        getattr(A.W, n).data = new
    assert torch.equal(A.run(act).y, yb)
    for n, (old, _) in zip(WEIGHTS, kept):
        getattr(A.W, n).set_(old)
    assert torch.equal(A.run(act).y, ya)
    # away to the host and back, as weights are offloaded
    host = [getattr(A.W, n).cpu() for n in WEIGHTS]
    for n in WEIGHTS:
        getattr(A.W, n).untyped_storage().resize_(0)
    hole = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    for n, h in zip(WEIGHTS, host):
        t = getattr(A.W, n)
        t.untyped_storage().resize_(h.untyped_storage().nbytes())
        t.copy_(h)
    assert torch.equal(A.run(act).y, ya)
    del hole


@pytest.mark.parametrize("act", ACTS)
def test_outputs_swapped_in_place(act):
    A, _ = _pair()
    b = A.run(act)
    y, first = b.y.clone(), b.y.data
    b.y.data = torch.zeros_like(first)
    first.fill_(3.0)
    A.run(act, b)
    assert torch.equal(b.y, y) and (first == 3.0).all()


@pytest.mark.parametrize("act", ACTS)
def test_copies(act):
    A, B = _pair()
    ya, yb = A.run(act).y.clone(), B.run(act).y.clone()
    b = moe.Mx4Buffers(A.p, act=act)
    W = A.W
    for how in (copy.copy, copy.deepcopy, lambda h: pickle.loads(pickle.dumps(h))):
        A.W, c = how(W), how(b)
        assert torch.equal(A.run(act, c).y, ya)
        for n in WEIGHTS:
            setattr(A.W, n, getattr(B.W, n))
        assert torch.equal(A.run(act).y, yb)
        A.W = W
        assert torch.equal(A.run(act, b).y, ya)
