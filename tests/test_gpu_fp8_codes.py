"""The norm's and SiLU-and-mul's 8-bit codes within half of e4m3's own step at each value
(test_gpu_fp8_silu's bound, which test_fp8_code_check.py tries on the CPU), and the forms of
w4a16_rmsnorm that only the C entry point has: 16-bit and 8-bit rows in one call, and a
residual whose sum is not kept.
"""
import ctypes

import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8_rows import WIDTHS, f64, norm_error, rows
from test_gpu_fp8_silu import check

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16 = torch.float16, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_norm_codes(w4, H, dtype):
    M = 33
    x, r = rows(H + 40, M, H, dtype), rows(H + 41, M, H, dtype, 2.0)
    w = (rows(H + 42, 1, H, F16, 0.1)[0].float() + 1).to(dtype)
    v = ref.rmsnorm(f64(x) + f64(r), f64(w), EPS)
    q, s, _ = w4.w4a16_rmsnorm_fp8(x.to(DEV), w.to(DEV), residual=r.to(DEV), eps=EPS)
    check(q, s, v, f"H={H}", E=norm_error(H))


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_silu_codes(w4, N, dtype):
    x = rows(N + 50, 33, 2 * N, dtype, 2.0)
    q, s = w4.w4a16_fp8_quant(x.to(DEV), epilogue=w4.EPILOGUE_SILU_MUL)
    check(q, s, ref.silu_mul(f64(x)), f"N={N}")


@pytest.mark.parametrize("H", [1, 129, 1024, 5119, 5120])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_norm_forms_of_the_c_entry_point(w4, H, dtype):
    M, G = 6, ref.groups(H)
    x, r = rows(H, M, H, dtype).to(DEV), rows(H + 1, M, H, dtype, 2.0).to(DEV)
    w = (rows(H + 2, 1, H, F16, 0.1)[0].float() + 1).to(dtype).to(DEV)
    code = w4.DTYPE_F16 if dtype == F16 else w4.DTYPE_BF16

    def call(res, total, y, q, s):
        p = [None if t is None else t.data_ptr() for t in (res, total, y, q, s)]
        assert w4.lib.w4a16_rmsnorm(x.data_ptr(), p[0], w.data_ptr(), M, H, ctypes.c_float(EPS),
                                    code, p[1], p[2], p[3], p[4],
                                    torch.cuda.current_stream().cuda_stream) == w4.W4A16_OK

    def fresh():
        return (torch.full((M, H), 7.0, dtype=dtype, device=DEV),
                torch.full((M, H), 7.0, dtype=dtype, device=DEV),
                torch.full((M, H), 7, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                torch.full((M, G), 7.0, device=DEV))

    for res in (None, r):
        y16 = w4.w4a16_rmsnorm(x, w, residual=res, eps=EPS)
        q8 = w4.w4a16_rmsnorm_fp8(x, w, residual=res, eps=EPS)
        want_y, want_h = y16 if res is not None else (y16, None)

        def same(y, q, s, h):
            assert y is None or torch.equal(y, want_y)
            assert q is None or (torch.equal(q.view(torch.uint8), q8[0].view(torch.uint8)) and
                                 torch.equal(s, q8[1]))
            assert h is None or torch.equal(h, want_h)

        h, y, q, s = fresh()
        call(res, None, y, q, s)          # both kinds of rows, no sum
        same(y, q, s, None)
        h, y, q, s = fresh()
        call(res, None, y, None, None)    # 16-bit rows alone, no sum
        same(y, None, None, None)
        h, y, q, s = fresh()
        call(res, None, None, q, s)       # 8-bit rows alone, no sum
        same(None, q, s, None)
        if res is not None:
            h, y, q, s = fresh()
            call(res, h, y, q, s)         # everything
            same(y, q, s, h)
            h.copy_(res)
            call(h, h, y, q, s)           # and in place of the residual
            same(y, q, s, h)
