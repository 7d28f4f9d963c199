"""The choice of experts (w4a16_moe_route) by sigmoids of logits far below zero, where
1 + e^-l leaves fp32's range: the weights are e^l to fp32's last bits, and renormalised
ones their shares.  Below l = -745, where binary64 has no e^l either, a weight is 0 (a mask
of the type's lowest value).  Tolerance: test_gpu_moe_route.py's, and its derivation (an exponential
of a difference d, one more of the logit itself, and quotients).
"""
import pytest
import torch

from test_gpu_moe_route import check

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("low,high", [(-92, -85), (-110, -80), (-300, -100), (-100, -10),
                                      (-95, 5), (-1e4, -1e3)])
def test_very_negative_logits(w4, low, high, dtype):
    g = torch.Generator().manual_seed(-int(low))
    logits = (low + (high - low) * torch.rand((40, 61), generator=g)).to(dtype).to(DEV)
    for k in (1, 2, 8):
        check(w4, logits, k, w4.ROUTE_SIGMOID, True)
        check(w4, logits, k, w4.ROUTE_SIGMOID, False)
    check(w4, logits, 5, w4.ROUTE_SIGMOID, True, scale=2.5)


def test_two_logits(w4):
    logits = torch.tensor([[-90.0, -91.0], [-700.0, -700.5], [-88.5, -float("inf")]], device=DEV)
    ids, weights = w4.w4a16_moe_route(logits, 2, scoring=w4.ROUTE_SIGMOID, renormalize=True)
    share = torch.tensor([1.0, 0.5]).exp() / (1 + torch.tensor([1.0, 0.5]).exp())
    assert torch.equal(ids.cpu(), torch.tensor([[0, 1]] * 3, dtype=torch.int32))
    assert torch.allclose(weights[:2, 0].cpu(), share, rtol=1e-6)
    assert weights[2].tolist() == [1.0, 0.0]


@pytest.mark.parametrize("renormalize", [True, False])
def test_rows_with_infinities_among_very_negative_logits(w4, renormalize):
    inf = float("inf")
    logits = torch.full((6, 40), -200.0)
    logits[0, 3] = inf
    logits[1, 2:] = -inf
    logits[2] = -inf
    logits[3, ::2] = float("nan")
    logits[4, 7] = 0.0
    logits[5, 1:4] = inf
    check(w4, logits.to(DEV), 6, w4.ROUTE_SIGMOID, renormalize)
