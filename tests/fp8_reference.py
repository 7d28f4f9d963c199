"""The 8-bit layer path in binary64 numpy, from its definition, for the tests:
e4m3 codes and their values, rows and weights in 8 bits, the linear, the norm
and silu-and-mul.  Shares no code with the package.
"""
import numpy as np
import torch

GROUP = 128
FLOOR = 2.0 ** -100


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes, from the format's definition."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v = np.nan
        elif e == 0:
            v = m / 8 * 2.0 ** -6
        else:
            v = (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = -v if c & 128 else v
    return t


TABLE = e4m3_table()
POSITIVE = TABLE[:127]  # ascending, 0 .. 448


def codes(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def values(t: torch.Tensor) -> np.ndarray:
    return TABLE[codes(t)]


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to the even code, by comparing with all of them."""
    a = np.minimum(np.abs(v), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, a), 1, 126)
    lo = hi - 1
    dlo, dhi = a - POSITIVE[lo], POSITIVE[hi] - a
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    return np.copysign(np.where(up, POSITIVE[hi], POSITIVE[lo]), v)


def groups(n: int) -> int:
    return -(-n // GROUP)


def row_scales(v: np.ndarray) -> np.ndarray:
    """Scales of rows v [M, N] (binary64): max(largest finite |v|, 2^-100) / 448."""
    M, N = v.shape
    a = np.zeros((M, groups(N) * GROUP))
    a[:, :N] = np.where(np.isfinite(v), np.abs(v), 0.0)
    return np.maximum(a.reshape(M, -1, GROUP).max(2), FLOOR) / 448.0


def expand(scales: np.ndarray, rows: int, M: int, N: int) -> np.ndarray:
    return scales.repeat(rows, 0)[:M].repeat(GROUP, 1)[:, :N]


def linear(x, xs, w, ws, residual=None):
    """(y, A) in binary64: y the result, A = sum |x| |w| (the scale of its sums)."""
    M, K = x.shape
    N = w.shape[0]
    X = values(x) * expand(xs.cpu().numpy().astype(np.float64), 1, M, K)
    W = values(w) * expand(ws.cpu().numpy().astype(np.float64), GROUP, N, K)
    with np.errstate(all="ignore"):
        y, A = X @ W.T, np.abs(X) @ np.abs(W).T
        if residual is not None:
            y = y + residual.detach().cpu().double().numpy()
    return y, A


def silu_mul(x: np.ndarray) -> np.ndarray:
    n = x.shape[1] // 2
    g, u = x[:, :n], x[:, n:]
    with np.errstate(all="ignore"):
        return g / (1 + np.exp(-g)) * u


def rmsnorm(h: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    with np.errstate(all="ignore"):
        return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


def make_linear(seed: int, M: int, N: int, K: int, dtype, residual: bool):
    """Seeded 8-bit operands (CPU): codes over the whole finite range, scales
    that differ from block to block, and a residual."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, K), generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    w = (torch.randn((N, K), generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    xs = torch.rand((M, groups(K)), generator=g) * 0.02 + 0.005
    ws = torch.rand((groups(N), groups(K)), generator=g) * 0.0005 + 0.0001
    r = (torch.randn((M, N), generator=g) * 4).to(dtype) if residual else None
    return x, xs, w, ws, r
