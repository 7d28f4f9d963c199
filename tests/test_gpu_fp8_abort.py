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


def test_counters_of_a_launch_cut_short_are_cleared_with_its_report(w4):
    # the probe leaves the workspace's first counter one too high: here that of a tile of 60
    # blocks that runs of 39 blocks cut in two, and of the first block of a 4-bit linear whose
    # K is split (each kernel would add up the pieces before the last one has come)
    M, N, K = 20, 12672, 7680
    x, xs, w, ws, _ = [None if t is None else t.to(DEV)
                       for t in ref.make_linear(73, M, N, K, torch.bfloat16, False)]
    N4, K4 = 5120, 17408
    x4 = torch.randn((4, K4), device=DEV).half()
    w4b = torch.randint(-2 ** 31, 2 ** 31, (N4, K4 // 8), device=DEV, dtype=torch.int64).int()
    s4 = torch.rand((N4, K4 // 128), device=DEV).half() * 0.01
    z4 = torch.randint(-2 ** 31, 2 ** 31, (N4, K4 // 1024), device=DEV, dtype=torch.int64).int()
    assert w4.w4a16_plan_info(4, N4, K4)["k_slices"] > 1

    def eight():
        return w4.w4a16_fp8_linear(x, xs, w, ws)

    def four():
        return w4.w4a16_linear(x4, w4b, s4, z4)

    for f in (eight, four):
        want = f()
        torch.cuda.synchronize()
        w4.w4a16_wait_probe()
        assert w4.w4a16_device_status() == 4096 | 8192
        for _ in range(3):
            assert torch.equal(f(), want)
    assert w4.w4a16_device_status() == 0
