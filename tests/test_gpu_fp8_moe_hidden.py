"""What the layer of 8-bit experts (w4a16_fp8_moe_mlp) keeps of h = silu(gate) up between
its two products: more bits than the 16-bit type has, a range that is not the 16-bit
type's, and silu's values far below zero.

The operands make gate and up exact: x and the codes are small whole numbers and the scales
powers of two, so that every sum is a whole number below 2^24 times one, and h's own error
is silu's (exponential and quotient, 2^-20) and what down takes of it, two bf16 values: each
rounds by at most 2^-8 of what is left, 2^-16 together.  Down adds a block's products and
blocks with (16 + G) 2^-22 of their magnitudes, the choices' sum rounds k + 2 times (2^-23),
and out once, by at most half a step u of its type.
"""
import numpy as np
import pytest
import torch

import fp8_reference
import routed_reference as ref

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


def silu(g):
    with np.errstate(all="ignore"):
        return g / (1 + np.exp(-g))


def definition(ops, dtype):
    """(out, bound), both [T, N], for operands with exact gates and ups."""
    x, ids, weights, w1, s1, w2, s2 = ops
    X, ids, wts = ref.f64(x), ids.numpy(), ref.f64(weights)
    (T, k), (_, N, I) = ids.shape, w2.shape
    out, off, size = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, N))
    c = (16 + fp8_reference.groups(I)) * 2.0 ** -22
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        both = X[t] @ ref.weight(w1[e], s1[e]).T
        h, W2 = silu(both[:, :I]) * both[:, I:], ref.weight(w2[e], s2[e])
        y, mag = h @ W2.T, np.abs(h) @ np.abs(W2).T
        wt = wts[t, j][:, None]
        np.add.at(out, t, wt * y)
        np.add.at(off, t, np.abs(wt) * (2.0 ** -16 + 2.0 ** -20 + 1.1 * c) * mag)
        np.add.at(size, t, np.abs(wt * y))
    bound = (off + (k + 2) * 2.0 ** -23 * (size + off) + ref.UNIT[dtype] * (np.abs(out) + off)
             + 2.0 ** -24)
    return out, bound


def operands(seed, T, k, E, K, I, N, dtype, gate=0.0625, up=0.0625, down=0.0625):
    g = torch.Generator().manual_seed(seed)

    def whole(shape, most):
        return torch.randint(-most, most + 1, shape, generator=g)

    def scales(rows, cols, s):
        return torch.full((E, fp8_reference.groups(rows), fp8_reference.groups(cols)), s)

    x = whole((T, K), 3).to(dtype)
    ids = torch.rand((T, E), generator=g).topk(k, 1).indices.to(torch.int32)
    weights = torch.ones((T, k)) / k
    w1 = whole((E, 2 * I, K), 3).float().to(torch.float8_e4m3fn)
    s1 = scales(2 * I, K, gate)
    if up != gate:  # by whole blocks of 128 rows
        assert I % 128 == 0
        s1[:, I // 128:] = up
    w2 = whole((E, N, I), 7).float().to(torch.float8_e4m3fn)
    return x, ids, weights, w1, s1, w2, scales(N, I, down)


def check(w4, ops, dtype):
    out = ref.f64(w4.w4a16_fp8_moe_mlp(*[t.to(DEV) for t in ops]))
    want, bound = definition(ops, dtype)
    assert np.isfinite(want).all()
    err = np.abs(out - want)
    bad = np.argwhere(~(err <= bound))
    assert bad.size == 0, (len(bad), bad[:3].tolist(), float(np.nanmax(err / bound)))
    assert w4.w4a16_device_status() == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,k,E,K,I,N", [(1, 1, 2, 64, 16, 4000), (2, 2, 4, 256, 32, 1021),
                                         (8, 2, 4, 128, 16, 1500), (12, 1, 1, 128, 32, 1200),
                                         (40, 2, 3, 256, 48, 600), (100, 2, 2, 128, 16, 400)])
def test_more_bits_than_the_16_bit_type(w4, T, k, E, K, I, N, dtype):
    check(w4, operands(T + I, T, k, E, K, I, N, dtype), dtype)


@pytest.mark.parametrize("T", [1, 6, 33])
def test_fp16_layers_beyond_65504(w4, T):
    # |h| to some 10^6 and 10^12, outputs of ordinary size
    check(w4, operands(T, T, 2, 3, 256, 128, 200, F16, gate=8.0, up=64.0, down=2.0 ** -20), F16)
    check(w4, operands(T + 1, T, 2, 3, 256, 128, 200, F16, gate=2.0 ** 10, up=2.0 ** 16,
                       down=2.0 ** -42), F16)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 6, 33])
def test_very_small_and_very_large(w4, T, dtype):
    check(w4, operands(T, T, 2, 3, 256, 128, 200, dtype, gate=0.0625, up=2.0 ** -70,
                       down=2.0 ** 66), dtype)
    check(w4, operands(T, T, 2, 3, 256, 128, 200, dtype, gate=0.0625, up=2.0 ** 105,
                       down=2.0 ** -109), dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_the_largest_finite_h(w4, dtype):
    # gate 64 (silu 64 to fp32's last bit) times the largest up below 2^122 is fp32's largest
    # number, whose nearest bf16 is Inf.  Codes of at most 1 keep down's own sum finite.
    K, I, N = 16, 128, 6
    x = torch.zeros((2, K))
    x[:, 0] = 1.0
    w1, w2 = torch.zeros((1, 2 * I, K)), torch.zeros((1, N, I))
    w1[0, 3, 0], w1[0, I + 3, 0] = 64.0, 1.0
    s1 = torch.ones((1, 2, 1))
    s1[0, 1, 0] = float(np.nextafter(np.float32(2.0 ** 122), np.float32(0)))
    codes = [1.0, -1.0, 0.5, 0.25, 0.0, -0.125]
    w2[0, :, 3] = torch.tensor(codes)
    f8 = torch.float8_e4m3fn
    ops = [x.to(dtype), torch.zeros((2, 1), dtype=torch.int32), torch.ones((2, 1)), w1.to(f8), s1,
           w2.to(f8), torch.full((1, 1, 1), 2.0 ** -120)]
    out = ref.f64(w4.w4a16_fp8_moe_mlp(*[o.to(DEV) for o in ops]))
    want = np.array(codes) * 64.0 * float(s1[0, 1, 0]) * 2.0 ** -120
    assert np.all(np.abs(out - want) <= (ref.UNIT[dtype] + 2.0 ** -15) * np.abs(want))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gates_far_below_zero(w4, dtype):
    """silu(g) = g e^g / (1 + e^g) does not vanish where 1 + e^-g leaves fp32's range: up is
    large there, and exact, as every sum has one product."""
    gates = [-30.0, -60.0, -80.0, -88.0, -96.0, -104.0, -112.0, -128.0, -144.0, -160.0]
    T, K, I, N = len(gates), 256, 128, 4
    x = torch.zeros((T, K))
    x[:, 0] = torch.tensor(gates) / -2.0  # (exact in both types)
    x[:, 200] = 1.0
    w1 = torch.zeros((1, 2 * I, K))
    w1[0, :I, 0] = -2.0
    w1[0, I:, 200] = 1.0
    s1 = torch.ones((1, 2, 2))
    w2 = torch.zeros((1, N, I))
    w2[0, 0, 5], w2[0, 1, 100], w2[0, 2, :2] = 1.0, -2.0, 0.5
    ops = [x.to(dtype), torch.zeros((T, 1), dtype=torch.int32), torch.ones((T, 1)),
           w1.to(torch.float8_e4m3fn), s1, w2.to(torch.float8_e4m3fn), torch.ones((1, 1, 1))]
    for t, g in enumerate(gates):
        # up so that h is near 1 (or as large as up can be)
        up = 2.0 ** min(126, int(-g / np.log(2)) - 4)
        s1[0, 1, 1] = up
        out = ref.f64(w4.w4a16_fp8_moe_mlp(*[o.to(DEV) for o in ops]))[t]
        h = g * np.exp(g) / (1 + np.exp(g)) * up
        want = h * np.array([1.0, -2.0, 1.0, 0.0])
        bound = (ref.UNIT[dtype] + 2.0 ** -15) * np.abs(want) + 2.0 ** -24
        assert np.all(np.abs(out - want) <= bound), (g, out, want)
    # -Inf is NaN, as in the quotient, and the other rows keep their bits (those of gates near
    # zero times this up are beyond fp16's range)
    before = w4.w4a16_fp8_moe_mlp(*[o.to(DEV) for o in ops]).cpu()
    ops[0][3, 0] = float("inf")
    out = w4.w4a16_fp8_moe_mlp(*[o.to(DEV) for o in ops]).cpu()
    rows = [t for t in range(T) if t != 3]
    assert out[3, :3].isnan().all() and torch.equal(out[rows], before[rows])
