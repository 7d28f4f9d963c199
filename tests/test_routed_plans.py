"""How the products whose weights a row chooses cut their work, asked of the library without
a GPU: refusals, and what the plans say.
"""
import ctypes

import pytest

import __graft_entry__


@pytest.fixture(scope="module")
def w4():
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


def test_fp8_moe_plan_refusals(w4):
    L, info = w4.lib.w4a16_fp8_moe_plan_info, (ctypes.c_int32 * 6)()
    bad, un = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_UNSUPPORTED
    good = dict(T=2, k=2, E=4, K=128, I=64, N=96)

    def code(out=info, **kw):
        return L(*{**good, **kw}.values(), out)

    assert code() == w4.W4A16_OK
    for name in good:
        assert code(**{name: 0}) == bad
        assert code(**{name: -1}) == bad
    assert code(out=None) == bad
    assert code(K=136) == bad and code(I=72) == bad and code(K=(1 << 22) + 16) == bad
    assert code(E=1025) == un and code(T=513) == un and code(T=1 << 30, k=8) == un


def test_fp8_moe_plan(w4):
    for T, k, E, K, I, N in ((1, 8, 128, 2048, 768, 2048), (64, 8, 128, 2048, 768, 2048),
                             (1024, 1, 1, 16, 16, 1), (1, 1, 1, 1 << 22, 1 << 22, 1 << 22)):
        p = w4.w4a16_fp8_moe_plan_info(T, k, E, K, I, N)
        for nt, ks in (p["gate_up"], p["down"]):
            assert nt in (1, 2, 4) and ks in (1, 2, 4, 8)
        assert p["grid"] >= 2 and p["ctas_per_sm"] in (0, 2)


def test_lora_plan_refusals(w4):
    L, info = w4.lib.w4a16_lora_plan_info, (ctypes.c_int32 * 3)()
    bad, un = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_UNSUPPORTED
    for sizes in ((0, 1, 8, 1), (65536, 1, 8, 1), (1, 0, 8, 1), (1, 1, 0, 1), (1, 1, 12, 1),
                  (1, 1, 8, 0), (-1, 1, 8, 1)):
        assert L(*sizes, info) == bad
    assert L(1, 1, 8, 1, None) == bad
    for sizes in ((1, 1025, 8, 1), (1, 1, 136, 1), (1, 1, 8, 5)):
        assert L(*sizes, info) == un
    if w4.lib.w4a16_device_sm_count() == 0:
        assert L(1, 1, 8, 1, info) == w4.W4A16_ERR_NOT_INITIALIZED
