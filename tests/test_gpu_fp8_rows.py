"""GPU parity of w4a16_rmsnorm, w4a16_rmsnorm_fp8 and w4a16_fp8_quant with their
definition in binary64: widths from 1 to 32768, partial groups, rows that are
aligned to 2 bytes only, empty batches, all-zero, tiny and non-finite rows, the
residual's sum in place, other streams and graphs.

Tolerances.  fp32 arithmetic before the stores: of v = h rstd w, h rounds once,
the sum of squares has at most n / 8 + 16 additions in any one chain (n the row's
width: 8 elements a step in a thread's chain, then two trees), its relative error
at most (n / 8 / 32 + 16 + 4) 2^-24 with at least 32 threads, half of it in rstd,
and the reciprocal, root and two products round once each: |v' - v| <= E |v| with
E = (n / 512 + 16) 2^-23.  silu-and-mul: expf is within 2 ulp, its argument exact,
the sum, the quotient and the product round once: E = 8 x 2^-23.  16-bit outputs:
u |v| + E |v| (u = 2^-11 fp16, 2^-8 bf16), plus fp16's subnormal spacing.  Scales:
(E + 2^-23) relative.  Codes: q * scale may differ from v by half a step of e4m3
at v (2^-4 |v|, or half of 2^-9 scales below 2^-6) plus v's error.  The plain
quantisation has no arithmetic before the division, so it is compared bit for
bit with IEEE fp32 division and rounding.
"""
import numpy as np
import pytest
import torch

import fp8_reference as ref

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


def rows(seed, M, N, dtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn((M, N), generator=g) * spread
    t[:, ::61] *= 10
    return t.to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def norm_error(n):
    return (n / 512 + 16) * 2.0 ** -23


def check16(y, v, E, what):
    u, tiny = (2.0 ** -11, 2.0 ** -25) if y.dtype == F16 else (2.0 ** -8, 0.0)
    err = np.abs(f64(y) - v)
    assert np.all(err <= (u + E) * np.abs(v) + tiny), f"{what}: worst {err.max():.3e}"


def check8(q, scales, v, E, what):
    M, N = v.shape
    want = ref.row_scales(v)
    s = f64(scales)
    assert s.shape == want.shape
    assert np.all(np.abs(s - want) <= (E + 2.0 ** -23) * want), f"{what}: scales"
    S = ref.expand(s, 1, M, N)
    got = ref.values(q) * S
    half = np.maximum(np.abs(v) * 2.0 ** -4, S * 2.0 ** -10)
    err = np.abs(got - v)
    bad = np.argwhere(~(err <= half * (1 + 2.0 ** -20) + (E + 2.0 ** -22) * np.abs(v)))
    assert bad.size == 0, f"{what}: {len(bad)} codes off, first {bad[:3].tolist()}"


WIDTHS = [1, 7, 8, 16, 127, 128, 129, 136, 255, 256, 1000, 1001, 1023, 1024, 2048, 5120, 6144,
          8192, 8200, 8201, 16384, 17408, 32768]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype,residual", [(F16, False), (BF16, True)])
def test_rmsnorm(w4, H, dtype, residual):
    M = 5
    x, w = rows(H, M, H, dtype), (rows(H + 1, 1, H, F16, 0.1)[0].float() + 1).to(dtype)
    r = rows(H + 2, M, H, dtype, 4.0) if residual else None
    h = f64(x) + (f64(r) if residual else 0.0)
    v = ref.rmsnorm(h, f64(w), EPS)
    E = norm_error(H)
    rd = r.to(DEV) if residual else None
    got16 = w4.w4a16_rmsnorm(x.to(DEV), w.to(DEV), residual=rd, eps=EPS)
    got8 = w4.w4a16_rmsnorm_fp8(x.to(DEV), w.to(DEV), residual=rd, eps=EPS)
    y = got16[0] if residual else got16
    check16(y, v, E, f"y H={H}")
    check8(got8[0], got8[1], v, E, f"q H={H}")
    if residual:
        for s in (got16[1], got8[2]):
            # the fp32 sum of two 16-bit values, rounded once
            assert torch.equal(s.cpu(), (x.float() + r.float()).to(dtype))


@pytest.mark.parametrize("M", [1, 2, 63, 600, 4000])
@pytest.mark.parametrize("H", [640, 5120])
def test_rmsnorm_many_rows(w4, M, H):
    x, w = rows(M, M, H, BF16), torch.ones(H, dtype=BF16)
    r = rows(M + 1, M, H, BF16, 4.0)
    q, s, total = w4.w4a16_rmsnorm_fp8(x.to(DEV), w.to(DEV), residual=r.to(DEV), eps=EPS)
    v = ref.rmsnorm(f64(x) + f64(r), f64(w), EPS)
    check8(q, s, v, norm_error(H), f"M={M}")
    assert torch.equal(total.cpu(), (x.float() + r.float()).to(BF16))


def test_rmsnorm_in_place_sum(w4):
    x, r, w = rows(1, 9, 1032, F16), rows(2, 9, 1032, F16, 4.0), torch.ones(1032, dtype=F16)
    q, s, want = w4.w4a16_rmsnorm_fp8(x.to(DEV), w.to(DEV), residual=r.to(DEV))
    rd = r.to(DEV)
    q2, s2, total = w4.w4a16_rmsnorm_fp8(x.to(DEV), w.to(DEV), residual=rd, sum_out=rd)
    assert total is rd and torch.equal(rd, want)
    assert np.array_equal(ref.codes(q), ref.codes(q2)) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rmsnorm_of_zero_and_non_finite_rows(w4, dtype):
    H = 300
    x = rows(3, 6, H, dtype)
    x[0] = 0                      # eps alone under the root: zeros out
    x[1, 5] = float("inf")        # rstd 0: the Inf becomes NaN, the rest zeros
    x[2, 299] = float("nan")      # the whole row
    x[3] = torch.finfo(dtype).smallest_normal
    w = torch.ones(H, dtype=dtype)
    q, s = w4.w4a16_rmsnorm_fp8(x.to(DEV), w.to(DEV), eps=EPS)
    y = w4.w4a16_rmsnorm(x.to(DEV), w.to(DEV), eps=EPS)
    got, y, s = ref.values(q), f64(y), f64(s)
    assert np.all(got[0] == 0) and np.all(y[0] == 0)
    assert np.all(s[0] == np.float32(2.0 ** -100) / np.float32(448))
    for out in (got, y):
        assert np.isnan(out[1, 5]) and np.all(np.delete(out[1], 5) == 0)
        assert np.isnan(out[2]).all()
        assert np.isfinite(out[3:]).all()
    v = ref.rmsnorm(f64(x[3:]), f64(w), EPS)
    check8(q[3:], torch.from_numpy(s[3:]), v, norm_error(H), "finite rows beside them")


def ieee_rows8(x):
    """Codes and scales with IEEE fp32 arithmetic (numpy), for the plain quantisation."""
    v = x.float().numpy()
    M, N = v.shape
    pad = np.zeros((M, ref.groups(N) * 128), dtype=np.float32)
    pad[:, :N] = v
    g = pad.reshape(M, -1, 128)
    a = np.where(np.isfinite(g), np.abs(g), np.float32(0)).max(2)
    s = np.maximum(a, np.float32(2.0 ** -100)) / np.float32(448)
    with np.errstate(all="ignore"):
        q = (g / s[:, :, None]).astype(np.float32)
    q = ref.round_e4m3(np.where(np.isfinite(g), q, 0).astype(np.float64))
    return np.where(np.isfinite(g), q, np.nan).reshape(M, -1)[:, :N], s


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_plain_quant_is_ieee_division(w4, N, dtype):
    x = rows(N + 9, 37, N, dtype, 3.0)
    x[0] = 0
    x[1] *= 2.0 ** -12
    x[2, N // 2] = float("nan")
    x[3, N // 3] = -float("inf")
    q, s = w4.w4a16_fp8_quant(x.to(DEV))
    want_q, want_s = ieee_rows8(x)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(ref.values(q), want_q, equal_nan=True)


def test_plain_quant_of_every_16_bit_value(w4):
    # all finite fp16 patterns, and all bf16 ones whose groups stay in fp32's
    # normal range, in every group of a row with its own largest value
    for dtype in (F16, BF16):
        bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dtype)
        x = bits.view(-1, 512)
        q, s = w4.w4a16_fp8_quant(x.to(DEV))
        want_q, want_s = ieee_rows8(x)
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(ref.values(q), want_q, equal_nan=True)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_silu_mul_quant(w4, N, dtype):
    x = rows(N + 3, 11, 2 * N, dtype, 2.0)
    x[0] = 0
    q, s = w4.w4a16_fp8_quant(x.to(DEV), epilogue=w4.EPILOGUE_SILU_MUL)
    check8(q, s, ref.silu_mul(f64(x)), 8 * 2.0 ** -23, f"N={N}")


def test_silu_mul_of_large_gates(w4):
    # silu's ends: e^-g over and under fp32's range, and gates of +-Inf and NaN
    gate = torch.tensor([200.0, -200.0, 88.0, -88.0, -100.0, 30000.0, -30000.0, 0.0,
                         float("inf"), -float("inf"), float("nan")], dtype=F16)
    x = torch.zeros((gate.numel(), 256), dtype=F16)
    x[:, :128] = gate[:, None]
    x[:, 128:] = 2.0
    q, s = w4.w4a16_fp8_quant(x.to(DEV), epilogue=w4.EPILOGUE_SILU_MUL)
    got = ref.values(q) * f64(s)
    finite = ref.silu_mul(f64(x[:8]))
    assert np.all(np.abs(got[:8] - finite) <= np.abs(finite) * 2.0 ** -3 + 2.0 ** -100)
    assert np.isnan(got[8:]).all()


@pytest.mark.parametrize("lead", [1, 3, 8])
def test_rows_aligned_to_two_bytes(w4, lead):
    # slices that start inside an allocation: 2-byte, 6-byte and 16-byte offsets
    M, N = 7, 1024

    def at(t):
        buf = torch.zeros(lead + t.numel() + 8, dtype=t.dtype, device=DEV)
        v = buf[lead:lead + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    x, r, w = rows(1, M, N, BF16), rows(2, M, N, BF16), rows(3, 1, N, BF16)[0]
    want = w4.w4a16_rmsnorm_fp8(x.to(DEV), w.to(DEV), residual=r.to(DEV))
    got = w4.w4a16_rmsnorm_fp8(at(x), at(w), residual=at(r))
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    a, b = w4.w4a16_fp8_quant(x.to(DEV)), w4.w4a16_fp8_quant(at(x))
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("N", [129, 1001, 1024])
def test_nothing_is_written_outside_the_rows(w4, N):
    M = 6
    x = rows(5, M, N, F16).to(DEV)
    want = w4.w4a16_fp8_quant(x)
    for lead in (1, 16):
        qb = torch.full((lead + M * N + 32,), 0x55, dtype=torch.uint8, device=DEV)
        sb = torch.full((1 + want[1].numel() + 9,), 3.0, device=DEV)
        q = qb[lead:lead + M * N].view(torch.float8_e4m3fn).view(M, N)
        s = sb[1:1 + want[1].numel()].view(want[1].shape)
        w4.w4a16_fp8_quant(x, q=q, scales=s)
        assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8))
        assert torch.equal(s, want[1])
        assert (qb[:lead] == 0x55).all() and (qb[lead + M * N:] == 0x55).all()
        assert sb[0] == 3 and (sb[1 + s.numel():] == 3).all()


def test_empty_batch(w4):
    x, w = torch.empty((0, 256), dtype=F16, device=DEV), torch.ones(256, dtype=F16, device=DEV)
    assert w4.w4a16_rmsnorm(x, w).shape == (0, 256)
    q, s, t = w4.w4a16_rmsnorm_fp8(x, w, residual=x)
    assert q.shape == (0, 256) and s.shape == (0, 2) and t.shape == (0, 256)
    q, s = w4.w4a16_fp8_quant(x, epilogue=w4.EPILOGUE_SILU_MUL)
    assert q.shape == (0, 128) and s.shape == (0, 1)


def test_another_stream_and_a_graph(w4):
    x, w = rows(6, 33, 2048, BF16).to(DEV), torch.ones(2048, dtype=BF16, device=DEV)
    want = w4.w4a16_rmsnorm_fp8(x, w) + w4.w4a16_fp8_quant(x, epilogue=w4.EPILOGUE_SILU_MUL)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (w4.w4a16_rmsnorm_fp8(x, w, stream=s) +
           w4.w4a16_fp8_quant(x, epilogue=w4.EPILOGUE_SILU_MUL, stream=s))
    s.synchronize()
    outs = [torch.zeros_like(t.view(torch.uint8)) for t in want]
    views = [o.view(t.dtype).view(t.shape) for o, t in zip(outs, want)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.w4a16_rmsnorm_fp8(x, w, q=views[0], scales=views[1])
        w4.w4a16_fp8_quant(x, epilogue=w4.EPILOGUE_SILU_MUL, q=views[2], scales=views[3])
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, views):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_rows_past_a_32_bit_offset(w4):
    # 2.4e9 elements: the last rows against the same rows alone
    M, N = 65535, 36864
    x = torch.zeros((M, N), dtype=F16, device=DEV)
    tail = rows(8, 5, N, F16).to(DEV)
    x[-5:] = tail
    q, s = w4.w4a16_fp8_quant(x)
    want = w4.w4a16_fp8_quant(tail)
    assert torch.equal(q[-5:].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(s[-5:], want[1]) and (q[:-5].view(torch.uint8) == 0).all()
