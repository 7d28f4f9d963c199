"""The layer of 8-bit experts (w4a16_fp8_moe_mlp) in every way it cuts its products: the
sizes of each case are searched for by the cut that the library names for them, so that a
changed rule cannot empty one.  Odd N, K and I that fill no block of 128, experts with more
slots than a tile.  Tolerance: test_gpu_fp8_moe.py's, and its derivation.
"""
import random

import pytest
import torch

import routed_reference as ref
from test_gpu_fp8_moe import check, dev

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
CUTS = [(1, 1), (1, 2), (1, 4), (1, 8), (2, 1), (2, 2), (4, 1)]


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, 64 << 20)
    return w4


def sizes(w4, product, cut):
    """The smallest (T, k, E, K, I, N) of many with this cut of this product."""
    rng, found = random.Random(7), []
    for _ in range(30000):
        T, k = rng.choice([1, 2, 3, 5, 9, 13, 17, 24, 33, 40, 64, 100]), rng.choice([1, 2, 3, 4, 8])
        E = rng.choice([1, 2, 3, 5, 8, 16])
        K, I, N = 16 * rng.randint(4, 100), 16 * rng.randint(2, 80), 2 * rng.randint(10, 800) + 1
        if (k <= E and I % 128 and K % 128
                and w4.w4a16_fp8_moe_plan_info(T, k, E, K, I, N)[product] == cut):
            found.append((E * (2 * I * K + N * I), T, k, E, K, I, N))
    assert found, (product, cut)
    # (the smallest, and the smallest with experts of several tiles)
    many = [f for f in found if f[1] * f[2] / f[3] > 8 * cut[0]]
    return [min(s)[1:] for s in (found, many) if s]


@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("product", ["gate_up", "down"])
def test_two_ctas_share_an_sm(w4, product, cut):
    for size in sizes(w4, product, cut):
        assert w4.w4a16_fp8_moe_plan_info(*size)["ctas_per_sm"] == 2


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("product", ["gate_up", "down"])
def test_every_cut(w4, product, cut, dtype):
    for size in sizes(w4, product, cut):
        ops = ref.make_experts(sum(size), *size, dtype)
        out = w4.w4a16_fp8_moe_mlp(*dev(ops))
        check(out, *ref.experts(*ops, dtype))
        assert torch.equal(w4.w4a16_fp8_moe_mlp(*dev(ops)), out)
        assert w4.w4a16_device_status() == 0
