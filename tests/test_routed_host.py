"""Host-side checks of the choice of experts, the layers of 8-bit experts and the low-rank
adapters (no GPU needed): every refusal comes before any CUDA call, with the header's status codes, and
the binding checks shapes, types and devices before the library is called.
"""
import ctypes

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


def _lora(w4, x=A, a=2 * A, b=3 * A, sc=4 * A, ranks=None, ids=5 * A, M=2, K=128, N=96, L=4, R=16,
          parts=(64, 32), n=None, dtype=0, res=6 * A, y=7 * A, scratch=8 * A, nbytes=1 << 20):
    host = None if parts is None else (ctypes.c_int32 * len(parts))(*parts)
    return w4.lib.w4a16_lora(x, a, b, sc, ranks, ids, M, K, N, L, R, host,
                             len(parts or ()) if n is None else n, dtype, res, y, scratch, nbytes,
                             None)


def test_lora_codes(w4):
    bad, odd, un = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_MISALIGNED, w4.W4A16_ERR_UNSUPPORTED
    names = ("x", "a", "b", "sc", "ids", "y", "scratch")
    for name in names:
        assert _lora(w4, **{name: None}) == bad
    for name in ("K", "N", "L", "R"):
        assert _lora(w4, **{name: 0}) == bad
    assert _lora(w4, M=-1) == bad and _lora(w4, M=65536) == bad
    assert _lora(w4, K=132) == bad and _lora(w4, R=12) == bad and _lora(w4, K=(1 << 22) + 8) == bad
    assert _lora(w4, parts=None) == bad and _lora(w4, n=0) == bad
    assert _lora(w4, parts=(64, 31)) == bad and _lora(w4, parts=(96, 0)) == bad
    assert _lora(w4, parts=(2 ** 31 - 1, 97)) == bad
    assert _lora(w4, parts=(20, 20, 20, 20, 16)) == un
    assert _lora(w4, L=1025) == un and _lora(w4, R=136) == un
    assert _lora(w4, dtype=2) == bad
    assert _lora(w4, x=A + 8) == odd and _lora(w4, a=2 * A + 8) == odd
    assert _lora(w4, b=3 * A + 2) == odd and _lora(w4, sc=4 * A + 2) == odd
    assert _lora(w4, ids=5 * A + 1) == odd and _lora(w4, ranks=9 * A + 2) == odd
    assert _lora(w4, res=6 * A + 1) == odd and _lora(w4, y=7 * A + 1) == odd
    assert _lora(w4, scratch=8 * A + 4) == odd
    need = w4.lib.w4a16_lora_scratch_bytes(2, 4, 16, 2)
    assert need >= 2 * 2 * 16 * 4
    assert _lora(w4, nbytes=need - 1) == w4.W4A16_ERR_WORKSPACE
    for at in (A, 2 * A, 3 * A, 4 * A, 5 * A):
        assert _lora(w4, y=at) == bad and _lora(w4, scratch=at) == bad
    assert _lora(w4, ranks=9 * A, y=9 * A) == bad
    assert _lora(w4, y=6 * A + 2) == bad and _lora(w4, scratch=6 * A) == bad
    assert _lora(w4, scratch=7 * A) == bad
    assert _lora(w4, M=0, **{n: None for n in names}) == w4.W4A16_OK
    for wrong in ((0, 4, 16, 2), (2, 1025, 16, 2), (2, 4, 136, 2), (2, 4, 16, 5)):
        assert w4.lib.w4a16_lora_scratch_bytes(*wrong) == 0
    if w4.lib.w4a16_device_sm_count() == 0:
        assert _lora(w4, nbytes=need) == w4.W4A16_ERR_NOT_INITIALIZED
        assert _lora(w4, res=7 * A) == w4.W4A16_ERR_NOT_INITIALIZED  # in place
        assert _lora(w4, res=None) == w4.W4A16_ERR_NOT_INITIALIZED


def test_lora_scratch_holds_the_plan(w4):
    # 16 bytes, 8 per tile, 2 per row, then t: M x parts x R floats
    for M, L in ((1, 1), (1, 1024), (17, 3), (4096, 1024), (65535, 1)):
        tiles = min(M, L) + M // 128 + 1  # full ones and a rest per adapter, those without
        need = 16 + 8 * tiles + 2 * M + M * 2 * 16 * 4
        assert w4.lib.w4a16_lora_scratch_bytes(M, L, 16, 2) >= need


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
    b = torch.zeros((4, 96, 16)).half()
    with pytest.raises(ValueError, match="x must live on a CUDA device"):
        w4.w4a16_lora(x, torch.zeros((4, 16, 128)).half(), b, torch.ones(4), ids[0])
    with pytest.raises(ValueError, match="b must be a 3-D"):
        w4.w4a16_lora(x, torch.zeros((4, 16, 128)).half(), b[0], torch.ones(4), ids[0])
