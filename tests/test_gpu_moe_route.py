"""The choice of experts (w4a16_moe_route) against a stable sort and 64-bit weights: all
types of logits, both scorings, every kernel's number of experts, ties, infinities, NaN,
rows of which nothing is left.

Tolerance of a weight, relative, with d the distance of its logit from the row's largest:
d is rounded once (d 2^-24), expf is within 2 units in the last place (2^-22), the E terms
of the sum carry the same errors (their d e^-d is at most 0.37 each, their sum at least 1)
and are added in at most 37 steps (37 x 2^-24); the quotients, the chosen weights' sum (at
most 32 further terms) and the factor add 2^-24 each: (d + 0.4 E + 96) 2^-24.
"""
import numpy as np
import pytest
import torch

import routed_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


def check(w4, logits, k, scoring, renormalize, scale=1.0, got=None):
    ids, weights = got or w4.w4a16_moe_route(logits, k, scoring=scoring, renormalize=renormalize,
                                             scale=scale)
    want, p, d = ref.route(logits, k, scoring == w4.ROUTE_SIGMOID, renormalize, scale)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want)
    off = np.abs(ref.f64(weights) - p)
    assert np.all(off <= (d + 0.4 * logits.shape[1] + 96) * 2.0 ** -24 * np.abs(p) + 1e-44)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (2, 3, 3), (5, 31, 4), (33, 33, 32),
                                   (77, 61, 5), (64, 64, 2), (9, 65, 6), (16, 129, 10),
                                   (301, 257, 8), (7, 512, 16), (3, 513, 1), (4, 1024, 32),
                                   (4099, 256, 8)])
def test_matches_sort(w4, T, E, k, dtype):
    g = torch.Generator(device=DEV).manual_seed(T * 1000 + E)
    logits = (2 * torch.randn((T, E), generator=g, device=DEV)).to(dtype)
    for scoring in (w4.ROUTE_SOFTMAX, w4.ROUTE_SIGMOID):
        for renormalize in (False, True):
            check(w4, logits, k, scoring, renormalize)
    check(w4, logits, k, w4.ROUTE_SOFTMAX, True, scale=2.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k", [(8, 8), (61, 7), (160, 9), (700, 32)])
def test_ties_go_to_the_lowest_index(w4, E, k, dtype):
    g = torch.Generator(device=DEV).manual_seed(E)
    logits = torch.randint(-2, 3, (200, E), generator=g, device=DEV).to(dtype)
    logits[0] = 0.0
    logits[1, ::2], logits[1, 1::2] = -0.0, 0.0  # equal, whatever their sign
    for scoring in (w4.ROUTE_SOFTMAX, w4.ROUTE_SIGMOID):
        check(w4, logits, k, scoring, True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k", [(5, 5), (40, 6), (300, 12)])
def test_infinities_and_nan(w4, E, k, dtype):
    inf, nan = float("inf"), float("nan")
    logits = torch.randn((10, E), generator=torch.Generator().manual_seed(E))
    logits[0] = -inf                 # nothing left
    logits[1] = nan
    logits[2, 1:] = -inf             # one left, fewer than k
    logits[3, ::2] = nan
    logits[4, 3] = inf
    logits[5, 1:4] = inf             # equal shares
    logits[6] = inf
    logits[7] = torch.finfo(dtype).min  # a mask of the type's lowest value
    logits[8, 2:] = torch.finfo(dtype).min
    logits[9, 0], logits[9, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min
    logits = logits.to(dtype).to(DEV)
    for scoring in (w4.ROUTE_SOFTMAX, w4.ROUTE_SIGMOID):
        for renormalize in (False, True):
            check(w4, logits, k, scoring, renormalize)


def test_outputs_given_streams_and_graphs(w4):
    g = torch.Generator(device=DEV).manual_seed(5)
    logits = torch.randn((50, 128), generator=g, device=DEV)
    want = w4.w4a16_moe_route(logits, 8)
    room = torch.full((52, 8), -7, dtype=torch.int32, device=DEV)
    wroom = torch.full((52, 8), -7.0, device=DEV)
    got = w4.w4a16_moe_route(logits, 8, topk_ids=room[1:51], weights=wroom[1:51])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for t in (room, wroom):
        assert bool((t[0] == -7).all()) and bool((t[51] == -7).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.w4a16_moe_route(logits, 8, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = w4.w4a16_moe_route(logits, 8)
    logits.copy_(torch.randn((50, 128), generator=g, device=DEV))
    graph.replay()
    check(w4, logits, 8, w4.ROUTE_SOFTMAX, True, got=got)
    # an odd first address, and no rows at all
    odd = torch.randn(50 * 61 + 1, generator=g, device=DEV).to(torch.bfloat16)[1:].view(50, 61)
    check(w4, odd, 3, w4.ROUTE_SIGMOID, True)
    none = w4.w4a16_moe_route(logits[:0], 8)
    assert none[0].shape == (0, 8) and none[1].shape == (0, 8)
