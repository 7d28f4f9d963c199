"""silu(gate) * up to 8-bit rows (w4a16_fp8_quant) over the whole range of the gate,
against binary64: whole groups of one gate from -30 down to the type's lowest value,
beside ups of every size, and such gates among ordinary ones.

Tolerance of silu(g) u before the division by the scale: the exponential is within
2^-22 and enters once (g >= -80) or twice (its square root, below), the terms left out of
its correction are under 9e-9, and every other step rounds once: at most
(2 x 2 + 2 + 1.5 + 0.3) 2^-23 < E = 8 x 2^-23.  Scales: (E + 2^-23) relative.  Codes:
q * scale is off by at most half of e4m3's step at v, 2^(floor(log2 |v / s|) - 4) s
(2^-10 s under 2^-6 s), plus v's error and the scale's.
"""
import numpy as np
import pytest
import torch

import fp8_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16 = torch.float16, torch.bfloat16
E = 8 * 2.0 ** -23


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


def quant(w4, x):
    return w4.w4a16_fp8_quant(x.to(DEV), epilogue=w4.EPILOGUE_SILU_MUL)


def check(q, scales, v, what, E=E):
    """Codes and scales of rows v (binary64), whose own error is E, within the tolerance above."""
    want = ref.row_scales(v)
    s = scales.cpu().double().numpy()
    off = np.abs(s - want) / want
    assert np.all(off <= E + 2.0 ** -23), (
        f"{what}: scales off by {off.max() * 2 ** 23:.1f} x 2^-23 at row {off.max(1).argmax()}")
    S = ref.expand(s, 1, *v.shape)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(v) / S * (1 + 2.0 ** -18)))
    half = np.exp2(np.maximum(e, -6.0) - 4) * S
    err = np.abs(ref.values(q) * S - v)
    bad = np.argwhere(~(err <= half + (2 * E + 2.0 ** -22) * np.abs(v)))
    assert bad.size == 0, f"{what}: {len(bad)} codes off, first {bad[:3].tolist()}"


GATES = {
    F16: [-30, -33, -40, -47, -55, -60, -72, -79.5, -79.9375, -80, -80.0625, -81, -85, -87.25,
          -87.5, -88, -88.75, -89, -90, -96, -100, -104, -110, -130, -1000, -30000, -65504],
    BF16: [-30, -33, -40, -47, -55, -60, -72, -79.5, -80, -80.5, -81, -85, -87, -87.5, -88, -88.5,
           -89, -90, -96, -100, -104, -110, -120, -130, -150, -165, -170, -200, -1e3, -1e6, -1e10,
           -1e20, -2e32, -1e35, -1e38, float(torch.finfo(BF16).min)],
}
UPS = {F16: [2.0 ** -10, 1.0, 1000.0, 32000.0],
       BF16: [2.0 ** -30, 1.0, 2.0 ** 40, 1e30, 1.6e38]}


@pytest.mark.parametrize("n", [256, 130])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_whole_groups_of_very_negative_gates(w4, dtype, n):
    g = torch.Generator().manual_seed(n)
    gates, ups = torch.tensor(GATES[dtype]).to(dtype), UPS[dtype]
    for up in ups:
        x = torch.empty((gates.numel(), 2 * n), dtype=dtype)
        x[:, :n] = gates[:, None]
        x[:, n:] = ((torch.rand((gates.numel(), n), generator=g) + 1) * up *
                    torch.where(torch.rand((gates.numel(), n), generator=g) < 0.5, -1, 1)).to(dtype)
        assert x.isfinite().all()
        q, s = quant(w4, x)
        check(q, s, ref.silu_mul(x.double().numpy()), f"up {up}")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_the_lowest_gate_with_the_largest_up_is_zero(w4, dtype):
    lim = torch.finfo(dtype)
    for gate in (lim.min, -30000.0, -1000.0):
        x = torch.full((1, 256), gate, dtype=dtype)
        x[:, 128:] = lim.max
        x[:, 129::2] = lim.min
        q, s = quant(w4, x)
        assert np.all(ref.values(q) == 0)
        assert float(s[0, 0]) == np.float32(2.0 ** -100) / np.float32(448)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_very_negative_gates_beside_ordinary_ones(w4, dtype):
    n, rows = 384, 64
    g = torch.Generator().manual_seed(7)
    x = (torch.randn((rows, 2 * n), generator=g) * 3).to(dtype)
    deep = torch.tensor(GATES[dtype]).to(dtype)
    at = torch.rand((rows, n), generator=g) < 0.1
    y = x.clone()
    y[:, :n][at] = deep[torch.randint(len(deep), (int(at.sum()),), generator=g)]
    q, s = quant(w4, y)
    check(q, s, ref.silu_mul(y.double().numpy()), "mixed")
    # with ordinary ups such elements are nothing beside the others: codes and scales are
    # those of the same rows with zero gates in their place
    z = x.clone()
    z[:, :n][at] = 0
    qz, sz = quant(w4, z)
    assert torch.equal(s, sz) and np.array_equal(ref.values(q), ref.values(qz))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinite_and_nan_gates_beside_very_negative_ones(w4, dtype):
    x = torch.zeros((3, 512), dtype=dtype)
    x[:, :256] = -100.0
    x[:, 256:] = 3.0
    x[:, 100] = torch.tensor([float("inf"), -float("inf"), float("nan")]).to(dtype)
    x[:, 200] = 1.0
    q, s = quant(w4, x)
    got = ref.values(q)
    assert np.isnan(got[:, 100]).all() and np.isfinite(np.delete(got, 100, 1)).all()
    assert np.all(got[:, 200] == 448) and np.all(np.delete(got[:, 128:], 72, 1) == 0)
