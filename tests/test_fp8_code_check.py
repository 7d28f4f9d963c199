"""The bound that the 8-bit row tests hold codes to (test_gpu_fp8_silu.check), tried on the
CPU with rows quantised in binary64: right codes pass, and a neighbouring code in the place
of any right one fails unless the value lies at the tie between them.
"""
import numpy as np
import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8_silu import E, check


def quantised(v):
    s = ref.row_scales(v).astype(np.float32)
    S = ref.expand(s.astype(np.float64), 1, *v.shape)
    q = torch.from_numpy(ref.round_e4m3(v / S)).float().to(torch.float8_e4m3fn)
    return q, torch.from_numpy(s), S


def test_right_codes_pass_and_neighbours_fail():
    g = np.random.default_rng(1)
    v = g.standard_normal((8, 300)) * np.exp2(g.integers(-6, 6, (8, 1)).astype(np.float64))
    v[0] = 0
    q, s, S = quantised(v)
    check(q, s, v, "right")
    codes = q.view(torch.uint8).numpy().astype(int)
    margin = (2 * E + 2.0 ** -21) * np.abs(v)
    tried = 0
    for up in (1, -1):
        other = np.where((codes & 127) + up >= 0, codes + up, codes)  # of the same sign
        other = np.where((other & 127) == 127, codes, other)
        value = ref.TABLE[other] * S
        step = np.abs(value - ref.TABLE[codes] * S)
        clear = (other != codes) & (np.abs(value - v) > step / 2 + margin + 1e-12)
        # the bound is half of the step above v's binade: a neighbour across its lower end,
        # where the step below is half as wide, may be nearer than that
        clear &= ~((codes & 7 == 0) & (up < 0))
        for r, c in np.argwhere(clear)[::17]:
            bad = codes.copy()
            bad[r, c] = other[r, c]
            with pytest.raises(AssertionError):
                check(torch.from_numpy(bad.astype(np.uint8)).view(torch.float8_e4m3fn), s, v,
                      "neighbour")
            tried += 1
    assert tried > 150


def test_a_wrong_scale_fails():
    v = np.random.default_rng(2).standard_normal((2, 256))
    q, s, _ = quantised(v)
    bad = s * (1 + 2.0 ** -18)
    with pytest.raises(AssertionError, match="scales"):
        check(q, bad, v, "scale")
