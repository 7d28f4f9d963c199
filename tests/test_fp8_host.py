"""Host-side checks of the 8-bit layer path's entry points (no GPU needed):
every refusal comes before any CUDA call, with the header's status codes, and
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


def _lin(w4, x=A, xs=2 * A, w=3 * A, ws=4 * A, M=2, N=64, K=256, dtype=0, epi=0, r=None, y=5 * A):
    return w4.lib.w4a16_fp8_linear(x, xs, w, ws, M, N, K, dtype, epi, r, y, None)


def test_fp8_linear_codes(w4):
    bad, odd, un = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_MISALIGNED, w4.W4A16_ERR_UNSUPPORTED
    for name in ("x", "xs", "w", "ws", "y"):
        assert _lin(w4, **{name: None}) == bad
    assert _lin(w4, M=-1) == bad and _lin(w4, M=65536) == bad
    assert _lin(w4, N=0) == bad and _lin(w4, K=0) == bad and _lin(w4, K=24) == bad
    assert _lin(w4, K=(1 << 22) + 16) == bad
    assert _lin(w4, dtype=2) == bad and _lin(w4, dtype=-1) == bad
    assert _lin(w4, epi=3) == bad and _lin(w4, epi=-1) == bad
    assert _lin(w4, epi=w4.EPILOGUE_SILU_MUL) == un
    assert _lin(w4, epi=w4.EPILOGUE_RESIDUAL) == bad      # no residual
    assert _lin(w4, r=6 * A) == bad                       # a residual nobody adds
    assert _lin(w4, x=A + 8) == odd and _lin(w4, w=3 * A + 4) == odd
    assert _lin(w4, xs=2 * A + 2) == odd and _lin(w4, ws=4 * A + 1) == odd
    assert _lin(w4, y=5 * A + 1) == odd
    assert _lin(w4, epi=1, r=6 * A + 1) == odd
    # y over an input, or partly over the residual
    for over in (A, 2 * A, 3 * A, 4 * A):
        assert _lin(w4, y=over) == bad
    assert _lin(w4, epi=1, r=5 * A + 2) == bad
    # an empty batch needs neither pointers nor w4a16_init
    assert _lin(w4, M=0, x=None, xs=None, w=None, ws=None, y=None) == w4.W4A16_OK
    assert _lin(w4, M=0, K=24) == bad
    if w4.lib.w4a16_device_sm_count() == 0:
        assert _lin(w4) == w4.W4A16_ERR_NOT_INITIALIZED
        assert _lin(w4, epi=1, r=5 * A) == w4.W4A16_ERR_NOT_INITIALIZED  # in place
        assert _lin(w4, y=5 * A + 2, K=16, N=1) == w4.W4A16_ERR_NOT_INITIALIZED


def _norm(w4, x=A, r=None, w=2 * A, M=2, H=256, eps=1e-6, dtype=0, s=None, y=None, q=5 * A,
          sc=6 * A):
    return w4.lib.w4a16_rmsnorm(x, r, w, M, H, eps, dtype, s, y, q, sc, None)


def test_rmsnorm_codes(w4):
    bad, odd = w4.W4A16_ERR_INVALID_ARG, w4.W4A16_ERR_MISALIGNED
    assert _norm(w4, x=None) == bad and _norm(w4, w=None) == bad
    assert _norm(w4, M=-1) == bad and _norm(w4, M=65536) == bad and _norm(w4, H=0) == bad
    assert _norm(w4, H=32769) == w4.W4A16_ERR_UNSUPPORTED
    assert _norm(w4, eps=-1.0) == bad and _norm(w4, eps=float("nan")) == bad
    assert _norm(w4, dtype=2) == bad
    assert _norm(w4, q=None, sc=None) == bad               # no output
    assert _norm(w4, q=None) == bad and _norm(w4, sc=None) == bad
    assert _norm(w4, s=3 * A) == bad                       # a sum of one term
    assert _norm(w4, x=A + 1) == odd and _norm(w4, w=2 * A + 1) == odd
    assert _norm(w4, r=3 * A + 1) == odd and _norm(w4, r=3 * A, s=4 * A + 1) == odd
    assert _norm(w4, y=4 * A + 1) == odd and _norm(w4, sc=6 * A + 2) == odd
    assert _norm(w4, q=A) == bad and _norm(w4, sc=2 * A) == bad and _norm(w4, y=A + 2) == bad
    assert _norm(w4, q=5 * A, y=5 * A) == bad and _norm(w4, sc=5 * A) == bad
    assert _norm(w4, r=3 * A, s=3 * A + 2) == bad and _norm(w4, r=3 * A, s=A) == bad
    assert _norm(w4, M=0, x=None, w=None, q=None, sc=None) == w4.W4A16_OK


def test_fp8_quant_codes(w4):
    L, bad = w4.lib.w4a16_fp8_quant, w4.W4A16_ERR_INVALID_ARG
    ok = (A, 2, 256, 0, 0, 2 * A, 3 * A, None)

    def put(i, v):
        return L(*ok[:i], v, *ok[i + 1:])

    for i in (0, 5, 6):
        assert put(i, None) == bad
    assert put(1, -1) == bad and put(1, 65536) == bad and put(2, 0) == bad
    assert put(3, w4.EPILOGUE_RESIDUAL) == w4.W4A16_ERR_UNSUPPORTED
    assert put(3, 3) == bad and put(4, 2) == bad
    assert L(A, 2, 255, w4.EPILOGUE_SILU_MUL, 0, 2 * A, 3 * A, None) == bad  # no halves
    assert put(0, A + 1) == w4.W4A16_ERR_MISALIGNED
    assert put(6, 3 * A + 2) == w4.W4A16_ERR_MISALIGNED
    assert put(5, A + 16) == bad and put(6, A + 16) == bad and put(6, 2 * A + 4) == bad
    assert L(None, 0, 256, 0, 0, None, None, None) == w4.W4A16_OK


def test_binding_checks_before_the_call(w4):
    f8 = torch.float8_e4m3fn
    x, xs = torch.zeros((2, 256), dtype=f8), torch.zeros((2, 2))
    w, ws = torch.zeros((64, 256), dtype=f8), torch.zeros((1, 2))
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        w4.w4a16_fp8_linear(x, xs, w, ws)
    with pytest.raises(ValueError, match="256 columns"):
        w4.w4a16_fp8_linear(x, xs, w[:, :128], ws)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        w4.w4a16_fp8_linear(x, xs, w, ws, dtype=torch.float32)
    with pytest.raises(ValueError, match="2-D"):
        w4.w4a16_fp8_quant(torch.zeros(8, dtype=torch.float16))
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        w4.w4a16_fp8_quant(torch.zeros((2, 8)))
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        w4.w4a16_rmsnorm(torch.zeros((2, 8), dtype=torch.float16),
                         torch.zeros(8, dtype=torch.float16))
    assert ctypes.sizeof(ctypes.c_float) == 4
