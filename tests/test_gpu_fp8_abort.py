"""The 8-bit linear and the library's report of a wait that gave up: warps of one block
of which only some have given up agree at the barrier of split tiles (the probe's second
warp reports what only the first has seen; had they not agreed, its bit would be missing),
and calls that split tiles give the same bits after the report as before it.
"""
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, 64 << 20)
    return w4


# equal runs of blocks: up to 64 tokens and more
SPLIT = [(20, 20480, 2816), (300, 10240, 3328)]


def operands():
    return [[None if t is None else t.to(DEV)
             for t in ref.make_linear(71, M, N, K, torch.bfloat16, True)] for M, N, K in SPLIT]


def outputs(w4, ops):
    return [w4.w4a16_fp8_linear(*o[:4], residual=o[4], epilogue=w4.EPILOGUE_RESIDUAL) for o in ops]


def test_warps_agree_on_a_wait_that_gave_up(w4):
    ops = operands()
    want = outputs(w4, ops)
    torch.cuda.synchronize()
    assert w4.w4a16_device_status() == 0
    w4.w4a16_wait_probe()
    assert w4.w4a16_device_status() == 4096 | 8192
    for a, b in zip(want, outputs(w4, ops)):
        assert torch.equal(a, b)
    assert w4.w4a16_device_status() == 0
