"""Low-rank adapters (w4a16_lora) with infinite weights and infinite A x: each output is
what the definition gives, the infinity of its sign, or NaN where it adds infinities of
both signs or multiplies one by zero; finite ones keep the tolerance of the adapters'
tests, routed_reference.py's.
"""
import numpy as np
import pytest
import torch

import routed_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16 = torch.float16, torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, 64 << 20)
    return w4


def call(w4, ops, kw):
    k = {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    y = ref.f64(w4.w4a16_lora(*[t.to(DEV) for t in ops], **k))
    assert w4.w4a16_device_status() == 0
    return y


def check(y, ops, kw, dtype):
    """Elements whose definition is infinite or NaN; the others by the bound of the same
    call with zeros in the place of the infinities (which they do not meet)."""
    want, _ = ref.adapters(*ops, kw["parts"], kw["ranks"], kw["residual"], dtype)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(y[inf], want[inf])
    clean = [t if t.dtype == torch.int32 else torch.where(t.isinf(), torch.zeros_like(t), t)
             for t in ops]
    _, bound = ref.adapters(*clean, kw["parts"], kw["ranks"], kw["residual"], dtype)
    ok = np.isfinite(want)
    assert np.all(np.abs(y[ok] - want[ok]) <= bound[ok])
    return want


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("R", [8, 24, 40, 128])
@pytest.mark.parametrize("M,parts", [(1, (64, 32)), (37, (64, 32)), (37, (61, 35)),
                                     (150, (64, 32)), (150, (61, 35))])
def test_infinite_weights_in_b(w4, M, parts, R, dtype):
    ops, kw = ref.make_adapters(M + R, M, 128, parts, 2, R, dtype,
                                ids=torch.arange(M, dtype=torch.int32) % 2)
    b = ops[2]
    b[:, 3, 1] = INF
    b[:, 8, R - 1] = -INF
    b[:, 70, 2] = INF
    b[:, 71, 2], b[:, 71, 5] = INF, -INF
    b[1, 33, 0] = -INF
    want = check(call(w4, ops, kw), ops, kw, dtype)
    assert np.isinf(want).any() and (M < 37 or np.isnan(want).any())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [8, 136])
def test_ax_of_every_kind_meets_infinite_weights(w4, M, dtype):
    """A x exact in the 16-bit type, zero, tiny beside the row's largest, of either sign."""
    R, K, parts = 8, 64, (40, 24)
    ops, kw = ref.make_adapters(3, M, K, parts, 1, R, dtype, ids=torch.zeros(M, dtype=torch.int32),
                                residual=False)
    x, a, b = ops[:3]
    x.zero_(), a.zero_()
    for p in range(2):
        for r in range(R):
            a[0, p * R + r, r] = 1.0  # t[m, r] = x[m, r], exactly
    x[:, :R] = torch.tensor([1.0, -1.0, 0.0, 2.0 ** -14, -2.0 ** -14, 3.0, 0.1, -1000.0]).to(dtype)
    x[1] = 0.0                                            # a row of zeros
    x[2, :R] *= 2.0 ** -10
    x[3, 7] = 2.0 ** 13 if dtype == F16 else 2.0 ** 100    # far from the others
    x[4, 3], x[4, 4] = torch.finfo(dtype).tiny, -torch.finfo(dtype).tiny
    for n in range(R):
        b[0, n, n], b[0, 8 + n, n] = INF, -INF            # each r alone
    b[0, 20, 0], b[0, 20, 1] = INF, INF                   # of both signs
    b[0, 21, 0], b[0, 21, 1] = INF, -INF
    b[0, 50, 6] = -INF
    want = check(call(w4, ops, kw), ops, kw, dtype)
    # (the third r is 0 in every row, which an infinite weight makes NaN)
    assert np.isnan(want[0, 2]) and np.isinf(want[0, [0, 1, 3, 4, 5, 6, 7]]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [8, 136])
def test_infinite_ax_beside_large_finite_ones(w4, M, dtype):
    """Of a row of A x with an infinity the finite ones, beyond the 16-bit type's range too,
    keep their values."""
    R, K, parts = 8, 64, (32,)
    ops, kw = ref.make_adapters(4, M, K, parts, 1, R, dtype, ids=torch.zeros(M, dtype=torch.int32),
                                residual=False)
    x, a, b = ops[:3]
    x.zero_(), a.zero_()
    for r in range(1, R):
        a[0, r, r] = 256.0
    a[0, 0, 0] = INF
    x[:, :R] = torch.tensor([3.0, -1000.0, 500.0, 0.5, -2.0, 700.0, -900.0, 1.0]).to(dtype)
    x[1::2, 0] = -3.0
    b[0, 3] = torch.tensor([1.0, 1, -1, 1, 1, -1, -1, 1]).to(dtype)   # Inf and finite ones
    b[0, 4] = torch.tensor([-1.0, 1, 1, 1, 1, 1, 1, 1]).to(dtype)
    b[0, 5] = torch.tensor([INF, -INF, 1, 1, 1, 1, 1, 1]).to(dtype)   # Inf Inf, + finite Inf
    b[0, 6] = torch.tensor([-INF, 1, 1, 1, 1, 1, 1, 1]).to(dtype)
    b[0, 7] = torch.tensor([0.0, 1, 1, 1, 1, 1, 1, 1]).to(dtype)      # 0 Inf
    b[0, 8] = torch.tensor([INF, 0, 0, 0, 0, 0, 0, 0]).to(dtype)
    y = call(w4, ops, kw)
    want, _ = ref.adapters(*ops, kw["parts"], None, None, dtype)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    inf = np.isinf(want)
    assert inf[:, 3].all() and np.isnan(want[1, 5]) and np.isnan(want[:, 7]).all()
    assert np.array_equal(y[inf], want[inf])
