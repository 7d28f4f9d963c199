"""GPU parity of the 8-bit linear (w4a16_fp8_linear) with its definition in
binary64: token counts on both sides of every tile size, ragged N, K whose last
block is partial, split and whole tiles, both output types, the residual (in
place too), exact integer cases, NaN and Inf operands, guards around the output,
other streams, graphs, small workspaces.

Tolerance, per element, with u the unit roundoff of the output type (2^-11 for
fp16, 2^-8 for bf16), G the blocks along K and A = sum |x| |w| over the element's
products (scales included):

    |y - ref| <= u |ref| + (16 + G) 2^-22 A + tiny

The one rounding of y gives the first term (and fp16's subnormal spacing, 2^-24,
gives tiny).  The products are exact in fp32; a block's sum comes from four
instructions that add 32 products each to the accumulator, every addition off by
at most one unit of the largest term (2^-23 A in total per instruction, doubled
for a truncating adder: 4 x 2^-22 A); a block's scale product and its
multiply-add round once each (2^-23 A), and so do the sums over G blocks
(2^-24 A each) and over the pieces of a split tile (at most G of them).
"""
import numpy as np
import pytest
import torch

import fp8_reference as ref

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


@pytest.fixture(autouse=True)
def no_device_errors(request):
    yield
    if "w4" in request.fixturenames:
        import weight_only_int4_w4a16_gb300 as w4
        assert w4.w4a16_device_status() == 0, "a kernel reported an expired bounded wait"


def bound(y_ref, A, K, dtype):
    u = 2.0 ** -11 if dtype == F16 else 2.0 ** -8
    return u * np.abs(y_ref) + (16 + ref.groups(K)) * 2.0 ** -22 * A + 2.0 ** -24


def check(y, want, A, K, what):
    got = y.detach().cpu().double().numpy()
    assert got.shape == want.shape
    err, tol = np.abs(got - want), bound(want, A, K, y.dtype)
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, (f"{what}: {len(bad)} of {want.size} off, first {bad[:3].tolist()}, "
                           f"worst {np.nanmax(err / tol):.2f} of the bound")


def call(w4, ops, dtype, y=None, **kw):
    x, xs, w, ws, r = [None if t is None else t.to(DEV) for t in ops]
    return w4.w4a16_fp8_linear(x, xs, w, ws, dtype=dtype, residual=r, y=y,
                               epilogue=w4.EPILOGUE_NONE if r is None else w4.EPILOGUE_RESIDUAL,
                               **kw)


SHAPES = [
    # one token, the smallest sizes, partial blocks of N and K
    (1, 1, 16), (1, 128, 128), (2, 17, 32), (1, 1024, 512), (1, 8192, 5120), (5, 48, 2064),
    # both sides of each tile of tokens
    (15, 129, 144), (16, 128, 256), (17, 255, 1040), (32, 1000, 528), (33, 1021, 1040),
    (64, 256, 4096), (65, 130, 272), (96, 640, 896), (127, 257, 384), (128, 384, 1152),
    (129, 1000, 528), (255, 513, 640), (256, 512, 512), (257, 768, 1296), (300, 520, 640),
    (513, 1153, 400), (1000, 1280, 768),
    # K long enough to be split many times; tiles in several waves
    (8, 5120, 17408), (64, 640, 17408), (3, 34816, 640), (200, 20000, 256), (700, 5120, 1024),
    (2000, 2304, 512),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,residual", [(BF16, False), (F16, True)])
def test_linear_matches_definition(w4, M, N, K, dtype, residual):
    ops = ref.make_linear(M * 7 + N + K, M, N, K, dtype, residual)
    y = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
    call(w4, ops, dtype, y=y)
    torch.cuda.synchronize()
    want, A = ref.linear(*ops)
    check(y, want, A, K, f"M={M} N={N} K={K}")


# one shape or two for every way the work is cut: up to 64 tokens, whole tiles, clusters
# of 2 .. 8 CTAs per tile, runs of blocks with tiles in two and three pieces; more
# tokens, whole tiles, clusters of 2, 3 and 4 pairs, whole tiles and then runs; each
# with rows that TMA can address (N a multiple of 8) and cannot, and with scale rows
# of whole 16-byte pieces (K / 128 a multiple of 4) and not
PLANS = [
    (2, 19456, 256), (2, 300, 384), (40, 384, 1152), (50, 1023, 2048), (7, 5120, 2304),
    (16, 9000, 1024), (5, 12800, 1280), (33, 12801, 1024), (64, 34816, 256),
    (70, 19456, 128), (128, 384, 1152), (512, 3840, 1024), (256, 5120, 1536), (256, 5121, 1664),
    (100, 704, 2048), (100, 701, 2048), (1100, 8200, 640), (1100, 8201, 512), (1100, 8202, 640),
    (900, 10240, 384),
    # long tiles in equal runs: the last wave would be mostly empty
    (3, 10300, 5648), (20, 20480, 2816), (50, 21001, 2704), (300, 10240, 3328), (500, 10241, 3216),
    # rows that TMA cannot address, split finely
    (123, 103, 944), (300, 1021, 1024), (200, 707, 528),
]


@pytest.mark.parametrize("M,N,K", PLANS)
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (F16, False)])
def test_every_way_to_cut_the_work(w4, M, N, K, dtype, residual):
    ops = ref.make_linear(M + N * 3 + K, M, N, K, dtype, residual)
    y = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
    call(w4, ops, dtype, y=y)
    again = call(w4, ops, dtype)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    want, A = ref.linear(*ops)
    check(y, want, A, K, f"M={M} N={N} K={K}")


@pytest.mark.parametrize("M,N,K", [(1, 200, 272), (20, 300, 1152), (130, 520, 640),
                                   (700, 1100, 528), (4, 1024, 8192)])
def test_integer_operands_are_exact(w4, M, N, K):
    # codes -2 .. 2 and scales that are powers of two: every product and sum is
    # a multiple of 2^-6 below 2^18, exact in fp32, so y is the exact value rounded once
    g = torch.Generator().manual_seed(K)
    x = torch.randint(-2, 3, (M, K), generator=g).float().to(torch.float8_e4m3fn)
    w = torch.randint(-2, 3, (N, K), generator=g).float().to(torch.float8_e4m3fn)
    xs = torch.exp2(torch.randint(-3, 1, (M, ref.groups(K)), generator=g).float())
    ws = torch.exp2(torch.randint(-3, 1, (ref.groups(N), ref.groups(K)), generator=g).float())
    r = torch.randint(-8, 9, (M, N), generator=g).to(BF16)
    for dtype in (F16, BF16):
        ops = (x, xs, w, ws, r.to(dtype))
        want, _ = ref.linear(*ops)
        y = call(w4, ops, dtype)
        assert torch.equal(y.cpu(), torch.from_numpy(want).float().to(dtype))


@pytest.mark.parametrize("M,N,K", [(3, 260, 4096), (64, 130, 528), (200, 400, 384), (600, 1000, 656)])
def test_residual_in_place(w4, M, N, K):
    ops = ref.make_linear(5, M, N, K, BF16, True)
    want = call(w4, ops, BF16)
    y = ops[4].to(DEV)
    x, xs, w, ws, _ = [t.to(DEV) for t in ops]
    got = w4.w4a16_fp8_linear(x, xs, w, ws, epilogue=w4.EPILOGUE_RESIDUAL, residual=y, y=y)
    assert got is y and torch.equal(y, want)


@pytest.mark.parametrize("M,N,K", [(2, 300, 2048), (40, 300, 400), (140, 300, 256), (600, 700, 256)])
def test_nan_and_inf_stay_in_their_row_and_column(w4, M, N, K):
    x, xs, w, ws, _ = ref.make_linear(11, M, N, K, F16, False)
    clean = call(w4, (x, xs, w, ws, None), F16).cpu()
    mi, ni = M // 2, N - 3
    codes = x.view(torch.uint8).clone()
    codes[mi, K - 1] = 0x7F  # NaN
    y = call(w4, (codes.view(torch.float8_e4m3fn), xs, w, ws, None), F16).cpu()
    rest = torch.arange(M) != mi
    assert y[mi].isnan().all() and torch.equal(y[rest], clean[rest])
    codes = w.view(torch.uint8).clone()
    codes[ni, 0] = 0xFF
    y = call(w4, (x, xs, codes.view(torch.float8_e4m3fn), ws, None), F16).cpu()
    rest = torch.arange(N) != ni
    assert y[:, ni].isnan().all() and torch.equal(y[:, rest], clean[:, rest])
    bad = xs.clone()
    bad[0, 0] = float("inf")
    y = call(w4, (x, bad, w, ws, None), F16).cpu()
    assert not y[0].isfinite().any() and torch.equal(y[1:], clean[1:])


@pytest.mark.parametrize("M,N,K", [(1, 77, 272), (31, 129, 144), (70, 131, 528), (300, 515, 400)])
def test_nothing_is_written_outside_the_output(w4, M, N, K):
    ops = ref.make_linear(21, M, N, K, BF16, False)
    want = call(w4, ops, BF16)
    for lead in (1, 8):  # y 2-byte aligned only, and 16-byte aligned
        buf = torch.full((lead + M * N + 64,), 7.0, dtype=BF16, device=DEV)
        y = buf[lead:lead + M * N].view(M, N)
        call(w4, ops, BF16, y=y)
        assert torch.equal(y, want)
        assert (buf[:lead] == 7).all() and (buf[lead + M * N:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(8, 5120, 17408), (48, 1000, 4096), (257, 1500, 2048),
                                   (1024, 2000, 1024)])
def test_runs_are_bit_identical(w4, M, N, K):
    ops = [None if t is None else t.to(DEV) for t in ref.make_linear(31, M, N, K, BF16, True)]
    ys = [call(w4, ops, BF16) for _ in range(6)]
    for y in ys[1:]:
        assert torch.equal(y.view(torch.int16), ys[0].view(torch.int16))


def test_back_to_back_shapes(w4):
    # launches that follow one another with other sizes, weights and workspaces
    cases = [(1, 1024, 512), (300, 520, 640), (8, 640, 8192), (65, 130, 272), (1, 1, 16),
             (1000, 1280, 768)]
    ops = [[None if t is None else t.to(DEV) for t in ref.make_linear(i, *c, F16, False)]
           for i, c in enumerate(cases)]
    alone = []
    for o in ops:
        alone.append(call(w4, o, F16))
        torch.cuda.synchronize()
    for _ in range(3):
        together = [call(w4, o, F16) for o in ops]
        for a, b in zip(alone, together):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(4, 2048, 5120), (600, 1300, 528)])
def test_another_stream_and_a_graph(w4, M, N, K):
    ops = [None if t is None else t.to(DEV) for t in ref.make_linear(41, M, N, K, BF16, False)]
    want = call(w4, ops, BF16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = call(w4, ops, BF16, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    y = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(w4, ops, BF16, y=y)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_empty_batch(w4):
    ops = ref.make_linear(51, 0, 64, 256, BF16, False)
    before = w4.w4a16_kernel_launches()
    assert call(w4, ops, BF16).shape == (0, 64)
    assert w4.w4a16_kernel_launches() == before


@pytest.mark.parametrize("M,N,K", [(8, 640, 8192), (100, 300, 4096), (400, 900, 2048)])
def test_a_small_workspace_splits_nothing(w4, M, N, K):
    ops = ref.make_linear(61, M, N, K, F16, True)
    want, A = ref.linear(*ops)
    w4.w4a16_init(0, 256)
    try:
        y = call(w4, ops, F16)
        torch.cuda.synchronize()
    finally:
        w4.w4a16_init(0, 64 << 20)
    check(y, want, A, K, "small workspace")


def test_more_tokens_than_a_32_bit_offset_reaches(w4):
    # y of 2.2e9 elements: rows past 2^31 elements against the same rows alone
    M, N, K = 63000, 34816, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randint(-8, 9, (M, K), generator=g, device=DEV).float().to(torch.float8_e4m3fn)
    w = torch.randint(-8, 9, (N, K), generator=g, device=DEV).float().to(torch.float8_e4m3fn)
    xs = torch.full((M, 1), 0.5, device=DEV)
    ws = torch.full((ref.groups(N), 1), 0.25, device=DEV)
    y = w4.w4a16_fp8_linear(x, xs, w, ws)
    tail = w4.w4a16_fp8_linear(x[-40:].contiguous(), xs[-40:].contiguous(), w, ws)
    assert torch.equal(y[-40:], tail)  # sums of multiples of 1/8: exact in any order
    mid = (1 << 31) // N
    part = w4.w4a16_fp8_linear(x[mid - 3:mid + 4].contiguous(), xs[:7].contiguous(), w, ws)
    assert torch.equal(y[mid - 3:mid + 4], part)
