"""How the 8-bit linear cuts its work, asked of the library without a GPU (152 SMs and
the default workspace are assumed): sizes at the ends of the accepted range, the rules of
the plans, refusals.
"""
import ctypes

import pytest

import __graft_entry__

MAX_N = 2 ** 31 - 1


@pytest.fixture(scope="module")
def w4():
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


@pytest.fixture(autouse=True)
def before_init(w4):
    if w4.lib.w4a16_device_sm_count() != 0:
        pytest.skip("w4a16_init has been called in this process: its workspace counts")


@pytest.mark.parametrize("N", [MAX_N, MAX_N - 126, MAX_N - 127, MAX_N - 255, 2 ** 31 - 256])
def test_weight_rows_near_the_largest_count(w4, N):
    p = w4.w4a16_fp8_plan_info(1, N, 16)
    assert p == {"wide": False, "grid": 152, "cluster_split": 1, "run_tiles": 0}
    p = w4.w4a16_fp8_plan_info(65, N, 16)
    assert p["wide"] and p["grid"] == 152 and p["cluster_split"] == 1


def test_rules(w4):
    def plan(*size):
        p = w4.w4a16_fp8_plan_info(*size)
        return p["wide"], p["grid"], p["cluster_split"], p["run_tiles"]

    assert plan(64, 34816, 256) == (False, 152, 1, 0)       # whole tiles, 272 of them
    assert plan(1, 128, 128) == (False, 1, 1, 0)            # one tile, one block
    assert plan(1, 8192, 5120) == (False, 128, 2, 0)        # 64 tiles, two CTAs each
    assert plan(8, 128, 4096) == (False, 8, 8, 0)           # one tile, eight CTAs
    assert plan(64, 20480, 5120) == (False, 152, 1, 160)    # 160 tiles in equal runs
    assert plan(65, 1024, 2048) == (True, 16, 2, 0)         # 4 tiles, two pairs each
    assert plan(300, 512, 4096) == (True, 32, 4, 0)         # 4 tiles, four pairs each
    assert plan(4096, 34816, 256) == (True, 152, 1, 0)
    assert plan(1000, 5120, 6144) == (True, 152, 1, 80)     # 80 tiles in equal runs


def test_refusals(w4):
    L, info = w4.lib.w4a16_fp8_plan_info, (ctypes.c_int32 * 4)()
    for size in ((0, 64, 64), (65536, 64, 64), (1, 0, 64), (1, 64, 0), (1, 64, 24),
                 (1, 64, (1 << 22) + 16), (-1, 64, 64), (1, -5, 64)):
        assert L(*size, info) == w4.W4A16_ERR_INVALID_ARG
    assert L(1, 64, 64, None) == w4.W4A16_ERR_INVALID_ARG
