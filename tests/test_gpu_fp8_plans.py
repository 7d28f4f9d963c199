"""The 8-bit linear in every way it cuts its work, each named by the plan that the
library gives for the sizes (so that a changed rule cannot empty a case): whole tiles,
clusters of 2 to 8 CTAs and of 2 to 4 pairs, equal runs with and without whole tiles
before them, with rows that TMA can address and cannot, with and without a residual; and
the workspace too small for equal runs.  Tolerance: test_gpu_fp8_linear's, and its
derivation.
"""
import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8_linear import check

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16 = torch.float16, torch.bfloat16
WORKSPACE = 64 << 20


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, WORKSPACE)
    return w4


def run(w4, M, N, K, dtype, residual, calls=3):
    ops = ref.make_linear(M + N * 3 + K, M, N, K, dtype, residual)
    x, xs, w, ws, r = [None if t is None else t.to(DEV) for t in ops]
    bits = None
    for _ in range(calls):
        y = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
        w4.w4a16_fp8_linear(x, xs, w, ws, dtype=dtype, residual=r, y=y,
                            epilogue=w4.EPILOGUE_NONE if r is None else w4.EPILOGUE_RESIDUAL)
        if bits is None:
            bits = y.view(torch.int16).clone()
        assert torch.equal(y.view(torch.int16), bits)
    want, A = ref.linear(*ops)
    check(y, want, A, K, f"M={M} N={N} K={K}")
    assert w4.w4a16_device_status() == 0


# sizes, then: the kernel of more than 64 tokens, a cluster's CTAs (pairs) per tile, tiles in
# equal runs
CASES = [
    # up to 64 tokens: 16, 32 and 64 at a time
    (3, 300, 128, False, 1, 0), (20, 34816, 256, False, 1, 0), (64, 20001, 272, False, 1, 0),
    (8, 8192, 2560, False, 2, 0), (20, 5121, 1040, False, 3, 0), (64, 4500, 1024, False, 4, 0),
    (40, 3500, 1280, False, 5, 0), (33, 2900, 1552, False, 6, 0), (12, 1025, 1808, False, 7, 0),
    (50, 1920, 4096, False, 8, 0),
    # equal runs shorter than a tile (two or three pieces each), and longer
    (16, 12672, 7680, False, 1, 99), (33, 12673, 7696, False, 1, 100),
    (20, 20480, 2816, False, 1, 160), (64, 20481, 2832, False, 1, 161),
    # more than 64
    (70, 300, 256, True, 1, 0), (1100, 8200, 640, True, 1, 0), (1100, 8201, 528, True, 1, 0),
    (300, 4608, 2048, True, 2, 0), (300, 4601, 528, True, 2, 0), (129, 5120, 3216, True, 3, 0),
    (200, 5119, 784, True, 3, 0), (512, 1024, 4096, True, 4, 0), (512, 1023, 1040, True, 4, 0),
    # all tiles in equal runs, and whole rounds before them
    (300, 10240, 6144, True, 1, 80), (300, 10241, 6144, True, 1, 82),
    (300, 10242, 6160, True, 1, 82), (1100, 8200, 6144, True, 1, 89),
    (1100, 8201, 6144, True, 1, 89), (1100, 8202, 6160, True, 1, 89),
]


@pytest.mark.parametrize("M,N,K,wide,cluster,runs", CASES)
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (F16, False)])
def test_every_plan(w4, M, N, K, wide, cluster, runs, dtype, residual):
    p = w4.w4a16_fp8_plan_info(M, N, K)
    assert (p["wide"], p["cluster_split"], p["run_tiles"]) == (wide, cluster, runs)
    run(w4, M, N, K, dtype, residual)


@pytest.mark.parametrize("M,N,K", [(20, 12672, 7680), (64, 20481, 2832), (300, 10241, 6144),
                                   (1100, 8200, 6144)])
def test_a_workspace_too_small_for_runs_leaves_tiles_whole(w4, M, N, K):
    assert w4.w4a16_fp8_plan_info(M, N, K)["run_tiles"] > 0
    w4.w4a16_init(0, 256)
    try:
        assert w4.w4a16_fp8_plan_info(M, N, K)["run_tiles"] == 0
        run(w4, M, N, K, BF16, True)
    finally:
        w4.w4a16_init(0, WORKSPACE)


def test_a_workspace_one_byte_short_of_the_pieces(w4):
    # what runs need: two slots per CTA of 128 rows by 16, 32 or 64 tokens, or two per pair of
    # 256 x 256, in 4 bytes each; the workspace comes in steps of 256
    sms = w4.lib.w4a16_device_sm_count()
    try:
        for (M, N, K), need in (((20, 12672, 7680), 2 * sms * 32 * 128 * 4),
                                ((300, 10241, 6144), 2 * (sms // 2) * 256 * 256 * 4)):
            w4.w4a16_init(0, need - 256)
            assert w4.w4a16_fp8_plan_info(M, N, K)["run_tiles"] == 0
            w4.w4a16_init(0, need)
            assert w4.w4a16_fp8_plan_info(M, N, K)["run_tiles"] > 0
            run(w4, M, N, K, F16, True)
    finally:
        w4.w4a16_init(0, WORKSPACE)
