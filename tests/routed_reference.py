"""The products whose weights a row chooses, in binary64 numpy, from their definitions,
for the tests: the choice of experts, layers of 8-bit experts, low-rank adapters.  Each
comes with the bound that its tests hold the kernels to, derived there.  Shares no code
with the package.
"""
import numpy as np
import torch

import fp8_reference as ref

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def route(logits: torch.Tensor, k: int, sigmoid: bool, renormalize: bool, scale: float = 1.0):
    """(ids [T, k], weights [T, k], d [T, k]): d the chosen logits' distance from the top."""
    z = f64(logits)
    z = np.where(np.isnan(z), -np.inf, z)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    chosen = np.take_along_axis(z, ids, 1)
    with np.errstate(all="ignore"):
        if sigmoid:
            p = 1 / (1 + np.exp(-chosen))
        else:
            top = z.max(1, keepdims=True)

            def share(v):
                return np.where(v == -np.inf, 0.0, np.where(v == top, 1.0, np.exp(v - top)))

            total = share(z).sum(1, keepdims=True)
            p = np.where(total > 0, share(chosen) / total, 0.0)
        # (no distance from an infinite logit: the p are exactly 0 or equal shares there)
        d = np.abs(chosen - z.max(1, keepdims=True))
        d = np.where(np.isfinite(d), d, 0.0)
        if renormalize:
            total = p.sum(1, keepdims=True)
            p = np.where(total > 0, p / total, 0.0)
    return ids, p * scale, d


def weight(w: torch.Tensor, s: torch.Tensor) -> np.ndarray:
    """One expert's weights [rows, cols] from its codes and its blocks' scales."""
    rows, cols = w.shape
    return ref.values(w) * ref.expand(f64(s), ref.GROUP, rows, cols)


def experts(x, ids, weights, w1, s1, w2, s2, dtype):
    """(out, bound), both [T, N]."""
    X, ids, wts = f64(x), ids.cpu().numpy(), f64(weights)
    T, k = ids.shape
    E, N, I = w2.shape
    u, K = UNIT[dtype], x.shape[1]
    c1, c2 = (16 + ref.groups(K)) * 2.0 ** -22, (16 + ref.groups(I)) * 2.0 ** -22
    out, off, size = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, N))
    with np.errstate(all="ignore"):
        for e in np.unique(ids[(ids >= 0) & (ids < E)]):
            t, j = np.nonzero(ids == e)
            W1, W2 = weight(w1[e], s1[e]), weight(w2[e], s2[e])
            both, A = X[t] @ W1.T, np.abs(X[t]) @ np.abs(W1).T
            g, up, dg, du = both[:, :I], both[:, I:], c1 * A[:, :I], c1 * A[:, I:]
            silu = g / (1 + np.exp(-g))
            h = silu * up
            dh = (1.1 * dg * (np.abs(up) + du) + np.abs(silu) * du
                  + (u + 2.0 ** -20) * np.abs(h) + 2.0 ** -24)
            y, mag = h @ W2.T, np.abs(h) @ np.abs(W2).T
            dy = dh @ np.abs(W2).T + c2 * (mag + dh @ np.abs(W2).T)
            c = wts[t, j][:, None]
            np.add.at(out, t, c * y)
            np.add.at(off, t, np.abs(c) * dy)
            np.add.at(size, t, np.abs(c * y))
        bound = off + (k + 2) * 2.0 ** -23 * (size + off) + u * (np.abs(out) + off) + 2.0 ** -24
    return out, bound


def make_experts(seed, T, k, E, K, I, N, dtype):
    """Seeded operands (CPU): distinct ids, codes over the whole finite range, scales that
    differ from block to block."""
    g = torch.Generator().manual_seed(seed)

    def codes(rows, cols):
        q = (torch.randn((E, rows, cols), generator=g) * 100).clamp(-448, 448)
        s = (0.5 + torch.rand((E, ref.groups(rows), ref.groups(cols)), generator=g))
        return q.to(torch.float8_e4m3fn), s * (cols ** -0.5 / 100)

    x = torch.randn((T, K), generator=g).to(dtype)
    ids = torch.rand((T, E), generator=g).topk(k, 1).indices.to(torch.int32)
    weights = torch.softmax(2 * torch.randn((T, k), generator=g), 1)
    return (x, ids, weights, *codes(2 * I, K), *codes(N, I))


def adapters(x, a, b, scales, ids, parts, ranks, residual, dtype):
    """(y, bound), both [M, N], of the low-rank adapters.

    With c = 2^-22 (16 + K / 16): t's K products (exact in fp32) are added 16 at a time, each
    addition off by a unit of the largest term (2^-23, doubled for a truncating adder), its
    slices and warps at most 16 + 16 times more.  t enters the second product with an error
    of 2^-16 (bf16: two roundings of 2^-8; fp16: 2^-22) of itself, and at least 2^-24 of the
    row's largest (fp16's subnormal spacing, as the row is scaled to at most 2).  Its sums
    over R carry 2^-22 (16 + R / 16) of their magnitudes, the factor and the sum with the
    residual three roundings, y one of its type.
    """
    X, S, ids = f64(x), f64(scales), ids.cpu().numpy()
    (M, K), (L, N, R), u = X.shape, b.shape, UNIT[dtype]
    y, off = np.zeros((M, N)), np.zeros((M, N))
    res = np.zeros((M, N)) if residual is None else f64(residual)
    adapted = np.zeros(M, dtype=bool)
    with np.errstate(all="ignore"):
        for l in range(L):
            rows = np.nonzero(ids == l)[0]
            r = R if ranks is None else min(max(int(ranks[l]), 0), R)
            if rows.size == 0 or r == 0:
                continue
            adapted[rows] = True
            first = 0
            for p, n in enumerate(parts):
                A, B = f64(a[l, p * R:p * R + r]), f64(b[l, first:first + n, :r])
                t, mag = X[rows] @ A.T, np.abs(X[rows]) @ np.abs(A).T
                dt = (2.0 ** -22 * (16 + K / 16) * mag + u * u * np.abs(t)
                      + 2.0 ** -24 * np.abs(t).max(1, keepdims=True))
                v, size = t @ B.T, (np.abs(t) + dt) @ np.abs(B).T
                dv = dt @ np.abs(B).T + (2.0 ** -22 * (16 + R / 16) + 3 * 2.0 ** -23) * size
                at = np.ix_(rows, np.arange(first, first + n))
                y[at], off[at] = S[l] * v, abs(S[l]) * dv
                first += n
        y = y + res
        bound = np.where(adapted[:, None],
                         off + 2.0 ** -23 * np.abs(res) + u * (np.abs(y) + off) + 2.0 ** -24, 0.0)
    return y, bound


def make_adapters(seed, M, K, parts, L, R, dtype, ids=None, ranks=False, residual=True):
    """Seeded operands (CPU) of the low-rank adapters, in the order of the call's arguments up
    to the ids, then a dict of the others."""
    g = torch.Generator().manual_seed(seed)
    N = sum(parts)
    x = torch.randn((M, K), generator=g).to(dtype)
    a = (torch.randn((L, len(parts) * R, K), generator=g) * K ** -0.5).to(dtype)
    b = (torch.randn((L, N, R), generator=g) * 0.5).to(dtype)
    scales = 0.5 + torch.rand(L, generator=g)
    if ids is None:
        ids = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    kw = dict(parts=list(parts),
              ranks=torch.randint(0, R + 1, (L,), generator=g, dtype=torch.int32) if ranks else None,
              residual=(torch.randn((M, N), generator=g) * 2).to(dtype) if residual else None)
    return (x, a, b, scales, ids), kw
