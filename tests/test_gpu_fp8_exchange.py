"""The 8-bit linear's exchange of a split tile's sums inside a cluster, for tiles whose
last tokens or columns do not exist: every output, nothing outside them, the same bits
in repeated calls.  Tolerance: test_gpu_fp8_linear's, and its derivation.
"""
import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8_linear import check

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, 64 << 20)
    return w4


SHAPES = [
    # many tokens, in clusters of 2 to 4 pairs of CTAs, 128 tokens per CTA and 32 per warp:
    # none in the second CTA, one or a few in a warp or a CTA, none in the last tile's second
    (65, 1024, 2048), (96, 1024, 2048), (100, 704, 2048), (128, 512, 3200), (129, 512, 2048),
    (161, 1024, 4096), (257, 1024, 2048), (300, 1024, 2048), (300, 1024, 4096), (385, 768, 2064),
    # columns: half a group of 16 (two pairs) at the edge, fewer columns than a CTA's part
    (300, 1032, 2048), (90, 1000, 2064), (70, 8, 4096), (300, 264, 2048), (257, 16, 2048),
    # the same in rows that TMA cannot address
    (100, 703, 2048), (300, 1021, 1024), (300, 1022, 4096), (65, 3, 4096), (385, 257, 528),
    # up to 64 tokens, in clusters of CTAs
    (1, 640, 4096), (3, 132, 2048), (17, 130, 2048), (33, 129, 4096), (63, 1021, 2048),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (F16, False)])
def test_split_tiles_with_an_edge(w4, M, N, K, dtype, residual):
    ops = ref.make_linear(M * 5 + N + K, M, N, K, dtype, residual)
    x, xs, w, ws, r = [None if t is None else t.to(DEV) for t in ops]
    want, A = ref.linear(*ops)
    bits = None
    for _ in range(4):
        buf = torch.full((8 + M * N + 64,), 7.0, dtype=dtype, device=DEV)
        y = buf[8:8 + M * N].view(M, N)
        w4.w4a16_fp8_linear(x, xs, w, ws, dtype=dtype, residual=r, y=y,
                            epilogue=w4.EPILOGUE_NONE if r is None else w4.EPILOGUE_RESIDUAL)
        assert (buf[:8] == 7).all() and (buf[8 + M * N:] == 7).all()
        if bits is None:
            bits = y.view(torch.int16).clone()
        assert torch.equal(y.view(torch.int16), bits)
    check(y, want, A, K, f"M={M} N={N} K={K}")
    assert w4.w4a16_device_status() == 0
