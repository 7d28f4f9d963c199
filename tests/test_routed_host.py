"""Host-side checks of the choice of experts and the layers of 8-bit experts (no GPU
needed): every refusal comes before any CUDA call, with the header's status codes, and
the binding checks shapes, types and devices before the library is called.
"""
import pytest
import torch

import __graft_entry__

A = 1 << 24  # a fake, 16-byte aligned "device address": never dereferenced on these paths


@pytest.fixture(scope="module")
def w4():
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


def _route(w4, l=A, T=2, E=64, k=8, dtype=0, scoring=0, renorm=1, scale=1.0, ids=2 * A, w=3 * A):
    return w4.lib.w4a16_moe_route(l, T, E, k, dtype, scoring, renorm, scale, ids, w, None)


def test_route_codes(w4):
    bad, odd, un = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_MISALIGNED, w4.W4A16_ERR_UNSUPPORTED
    for name in ("l", "ids", "w"):
        assert _route(w4, **{name: None}) == bad
    assert _route(w4, T=-1) == bad and _route(w4, T=65536) == bad and _route(w4, E=0) == bad
    assert _route(w4, k=0) == bad and _route(w4, k=65) == bad
    assert _route(w4, E=1025) == un and _route(w4, k=33) == un
    assert _route(w4, dtype=3) == bad and _route(w4, dtype=-1) == bad
    assert _route(w4, scoring=2) == bad and _route(w4, scoring=-1) == bad
    assert _route(w4, l=A + 1) == odd and _route(w4, l=A + 2, dtype=2) == odd
    assert _route(w4, ids=2 * A + 2) == odd and _route(w4, w=3 * A + 1) == odd
    assert _route(w4, ids=A) == bad and _route(w4, w=A + 4) == bad and _route(w4, w=2 * A) == bad
    assert _route(w4, T=0, l=None, ids=None, w=None) == w4.W4A16_OK


def _mlp(w4, x=A, ids=2 * A, wt=3 * A, T=2, k=2, E=4, K=128, I=64, N=96, dtype=0, w1=4 * A,
         s1=5 * A, w2=6 * A, s2=7 * A, out=8 * A, scratch=9 * A, nbytes=1 << 20):
    return w4.lib.w4a16_fp8_moe_mlp(x, ids, wt, T, k, E, K, I, N, dtype, w1, s1, w2, s2, out,
                                    scratch, nbytes, None)


def test_fp8_moe_codes(w4):
    bad, odd, un = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_MISALIGNED, w4.W4A16_ERR_UNSUPPORTED
    names = ("x", "ids", "wt", "w1", "s1", "w2", "s2", "out", "scratch")
    for name in names:
        assert _mlp(w4, **{name: None}) == bad
    for name in ("k", "E", "K", "I", "N"):
        assert _mlp(w4, **{name: 0}) == bad
    assert _mlp(w4, T=-1) == bad and _mlp(w4, K=136) == bad and _mlp(w4, I=72) == bad
    assert _mlp(w4, K=(1 << 22) + 16) == bad and _mlp(w4, dtype=2) == bad
    assert _mlp(w4, T=513) == un and _mlp(w4, T=1 << 30, k=8) == un and _mlp(w4, E=1025) == un
    assert _mlp(w4, x=A + 8) == odd and _mlp(w4, w1=4 * A + 4) == odd
    assert _mlp(w4, w2=6 * A + 8) == odd and _mlp(w4, scratch=9 * A + 8) == odd
    assert _mlp(w4, ids=2 * A + 2) == odd and _mlp(w4, wt=3 * A + 2) == odd
    assert _mlp(w4, s1=5 * A + 2) == odd and _mlp(w4, out=8 * A + 1) == odd
    need = w4.lib.w4a16_fp8_moe_scratch_bytes(2, 2, 64, 96)
    assert need >= 2 * 2 * (64 * 2 + 96 * 4)
    assert _mlp(w4, nbytes=need - 1) == w4.W4A16_ERR_WORKSPACE
    for at in (A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A):
        assert _mlp(w4, out=at) == bad and _mlp(w4, scratch=at) == bad
    assert _mlp(w4, out=9 * A) == bad
    assert _mlp(w4, T=0, **{n: None for n in names}) == w4.W4A16_OK
    assert w4.lib.w4a16_fp8_moe_scratch_bytes(0, 2, 64, 96) == 0
    assert w4.lib.w4a16_fp8_moe_scratch_bytes(513, 2, 64, 96) == 0
    if w4.lib.w4a16_device_sm_count() == 0:
        assert _mlp(w4, nbytes=need) == w4.W4A16_ERR_NOT_INITIALIZED
        assert _mlp(w4, T=512) == w4.W4A16_ERR_NOT_INITIALIZED


def test_binding_checks_before_the_call(w4):
    with pytest.raises(ValueError, match="logits must live on a CUDA device"):
        w4.w4a16_moe_route(torch.zeros((2, 8)), 2)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        w4.w4a16_moe_route(torch.zeros((2, 8), dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="2-D"):
        w4.w4a16_moe_route(torch.zeros(8), 2)
    f8 = torch.float8_e4m3fn
    x, ids, wt = torch.zeros((2, 128)).half(), torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2))
    w1, s1 = torch.zeros((4, 128, 128), dtype=f8), torch.zeros((4, 1, 1))
    w2, s2 = torch.zeros((4, 96, 64), dtype=f8), torch.zeros((4, 1, 1))
    with pytest.raises(ValueError, match="x must live on a CUDA device"):
        w4.w4a16_fp8_moe_mlp(x, ids, wt, w1, s1, w2, s2)
    with pytest.raises(ValueError, match="w_gate_up must be a 3-D"):
        w4.w4a16_fp8_moe_mlp(x, ids, wt, w1[0], s1, w2, s2)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        w4.w4a16_fp8_moe_mlp(x.float(), ids, wt, w1, s1, w2, s2)
