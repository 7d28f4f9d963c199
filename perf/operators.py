"""What is timed of the FP8 layer path: an RMS norm that writes 8-bit rows, the
8-bit quantisation of a layer's rows (plain, or of silu(gate) * up), and the
8-bit linear that reads them.

Data (e4m3 = 4 exponent and 3 mantissa bits, largest value 448):
  rows     q [M, K] e4m3 with scales [M, ceil(K/128)] fp32, one per 128
           consecutive elements of a row: the row is q * scale
  weights  w [N, K] e4m3 with scales [ceil(N/128), ceil(K/128)] fp32, one per
           block of 128 x 128

  norm     h = x + residual, v = h / sqrt(mean(h^2) + eps) * weight; the
           outputs are v (16 bits) or its rows in 8 bits, and h (16 bits)
  quant    v = x, or v = silu(x[:, :n]) * x[:, n:]; its rows in 8 bits
  linear   y = rows @ weights^T (+ residual), 16 bits

A group's scale is max(a, 2^-100) / 448 with a the largest finite magnitude of
the group; an element is v / scale rounded to e4m3 (nearest, ties to even), and
Inf and NaN become e4m3's NaN.

With ``own`` false, ``run`` computes this with elementary torch operations in
32 bits; with ``own`` true it makes the calls of this package.
"""
import functools
import math

import torch

own = False

GROUP = 128
E4M3_MAX = 448.0
FLOOR = 2.0 ** -100
EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # --- the 8-bit linear (the decode layer's four shapes and odd ones)
        # one token of plain decode through the fused qkv projection
        dict(name="linear m1 qkv", op="linear", M=1, N=8192, K=5120, dtype="bf16", residual=False),
        # a verify pass of 1 + 7 drafted tokens through gate+up
        dict(name="linear m8 gate_up", op="linear", M=8, N=34816, K=5120, dtype="f16",
             residual=False),
        # a ragged batch through a layer whose sizes are multiples of nothing
        dict(name="linear m37 odd", op="linear", M=37, N=1021, K=1040, dtype="bf16", residual=True),
        # the largest decode round's tokens through down, added to the stream
        dict(name="linear m64 down", op="linear", M=64, N=5120, K=17408, dtype="bf16",
             residual=True),
        # a short prompt through the attention's output projection
        dict(name="linear m1000 o", op="linear", M=1000, N=5120, K=6144, dtype="bf16",
             residual=True),
        # a prefill chunk through gate+up: the largest product of the layer
        dict(name="linear m4096 gate_up", op="linear", M=4096, N=34816, K=5120, dtype="bf16",
             residual=False),
        # --- the norm before qkv and gate+up
        # one decoded token: latency
        dict(name="norm m1 fp8", op="norm", M=1, N=5120, out="fp8", dtype="bf16", residual=True),
        # odd rows in 16 bits, for a layer whose weights are not in 8 bits
        dict(name="norm m77 odd", op="norm", M=77, N=1023, out="16", dtype="f16", residual=False),
        # a prefill of 8192 tokens
        dict(name="norm m8192 fp8", op="norm", M=8192, N=5120, out="fp8", dtype="bf16",
             residual=True),
        # --- the quantisation before down (silu(gate) * up) and o (plain)
        # a verify pass
        dict(name="quant silu m8", op="quant", M=8, N=17408, silu=True, dtype="f16"),
        # attention's output, a ragged batch and an odd width
        dict(name="quant m301 odd", op="quant", M=301, N=1001, silu=False, dtype="f16"),
        # a prefill chunk
        dict(name="quant silu m4096", op="quant", M=4096, N=17408, silu=True, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "quant"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "linear":
        while True:
            M = _spread(rng, 1, 8192)
            N = _spread(rng, 48, 34816)
            K = 16 * _spread(rng, 8, 1088)  # rows of whole 16-byte pieces
            if M * N * K <= 4096 * 34816 * 5120:
                break
        if rng.random() < 0.5:  # half of them in whole blocks, as layers mostly are
            N = -(-N // 128) * 128
            K = -(-K // 128) * 128
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, residual=rng.random() < 0.5)
    M = _spread(rng, 1, 8192)
    if op == "norm":
        N = _spread(rng, 64, 8192)
        if rng.random() < 0.5:
            N = -(-N // 128) * 128
        return dict(op=op, M=M, N=N, out=rng.choice(["fp8", "16"]), dtype=dtype,
                    residual=rng.random() < 0.5)
    while True:
        N = _spread(rng, 64, 17408)
        if M * N <= 4096 * 17408:
            break
    if rng.random() < 0.5:
        N = -(-N // 128) * 128
    return dict(op=op, M=M, N=N, silu=rng.random() < 0.5, dtype=dtype)


def work(case):
    M, N = case["M"], case["N"]
    groups = -(-N // GROUP)
    if case["op"] == "linear":
        K = case["K"]
        G = -(-K // GROUP)
        byte = M * K + 4 * M * G + N * K + 4 * groups * G + 2 * M * N * (2 if case["residual"] else 1)
        return {"bytes": byte, "flops": 2 * M * N * K}
    rows = M * N + 4 * M * groups  # q and its scales
    if case["op"] == "norm":
        byte = 2 * M * N * (3 if case["residual"] else 1) + 2 * N
        byte += rows if case["out"] == "fp8" else 2 * M * N
        return {"bytes": byte, "flops": 6 * M * N}
    return {"bytes": 2 * M * N * (2 if case["silu"] else 1) + rows,
            "flops": (10 if case["silu"] else 4) * M * N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, dtype, spread=1.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, spread, generator=gen)
    return t.to(dtype)


def _activations(gen, M, N, dtype):
    """Rows as a decoder's stream has them: about one column in 64 is ten times the others."""
    t = torch.empty((M, N), dtype=torch.float32, device="cuda").normal_(generator=gen)
    big = torch.rand(N, generator=gen, device="cuda") < 1.0 / 64
    return (t * torch.where(big, 10.0, 1.0)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    M, N = case["M"], case["N"]
    s = dict(case)
    if case["op"] == "linear":
        K = case["K"]
        s["x"], s["x_scales"] = _rows8(_activations(gen, M, K, torch.float32))
        s["w"], s["w_scales"] = _blocks8(_normal(gen, (N, K), torch.float32, 0.03))
        s["residual"] = _normal(gen, (M, N), dt, 4.0) if case["residual"] else None
        s["dt"] = dt
    elif case["op"] == "norm":
        s["x"] = _activations(gen, M, N, dt)
        s["residual"] = _normal(gen, (M, N), dt, 4.0) if case["residual"] else None
        s["weight"] = (1.0 + _normal(gen, (N,), torch.float32, 0.1)).to(dt)
    else:
        s["x"] = _activations(gen, M, 2 * N if case["silu"] else N, dt)
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _padded(v, rows, cols):
    return torch.nn.functional.pad(v, (0, -v.shape[1] % cols, 0, -v.shape[0] % rows))


def _rows8(v):
    """Rows v [M, N] fp32 -> (e4m3 [M, N], scales [M, ceil(N/128)])."""
    M, N = v.shape
    g = _padded(v, 1, GROUP).view(M, -1, GROUP)
    a = torch.where(torch.isfinite(g), g.abs(), 0.0).amax(-1)
    scale = a.clamp(min=FLOOR) / E4M3_MAX
    q = g / scale[:, :, None]
    q = torch.where(torch.isfinite(g), q, math.nan).reshape(M, -1)[:, :N]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def _blocks8(w):
    """Weights w [N, K] fp32 -> (e4m3 [N, K], scales [ceil(N/128), ceil(K/128)])."""
    N, K = w.shape
    b = _padded(w, GROUP, GROUP)
    nb, kb = b.shape[0] // GROUP, b.shape[1] // GROUP
    b = b.view(nb, GROUP, kb, GROUP)
    scale = b.abs().amax((1, 3)).clamp(min=FLOOR) / E4M3_MAX
    q = (b / scale[:, None, :, None]).reshape(nb * GROUP, kb * GROUP)[:N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def _expanded(scales, rows, cols, M, N):
    return scales.repeat_interleave(rows, 0)[:M].repeat_interleave(cols, 1)[:, :N]


def _plain(s):
    if s["op"] == "linear":
        M, K = s["x"].shape
        N = s["w"].shape[0]
        x = s["x"].float() * _expanded(s["x_scales"], 1, GROUP, M, K)
        w = s["w"].float() * _expanded(s["w_scales"], GROUP, GROUP, N, K)
        y = x @ w.t()
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(s["dt"])}
    x = s["x"].float()
    if s["op"] == "quant":
        if s["silu"]:
            n = s["N"]
            gate = x[:, :n]
            x = gate / (1.0 + torch.exp(-gate)) * x[:, n:]
        q, scales = _rows8(x)
        return {"q": q, "scales": scales}
    out = {}
    if s["residual"] is not None:
        x = x + s["residual"].float()
        out["sum"] = x.to(s["x"].dtype)
    v = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if s["out"] == "fp8":
        out["q"], out["scales"] = _rows8(v)
    else:
        out["y"] = v.to(s["x"].dtype)
    return out


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _package():
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(torch.cuda.current_device())
    return w4


def _call(s):
    w4 = _package()
    if s["op"] == "linear":
        res = s["residual"]
        return {"y": w4.w4a16_fp8_linear(
            s["x"], s["x_scales"], s["w"], s["w_scales"], dtype=s["dt"],
            epilogue=w4.EPILOGUE_NONE if res is None else w4.EPILOGUE_RESIDUAL, residual=res)}
    if s["op"] == "quant":
        q, scales = w4.w4a16_fp8_quant(
            s["x"], epilogue=w4.EPILOGUE_SILU_MUL if s["silu"] else w4.EPILOGUE_NONE)
        return {"q": q, "scales": scales}
    out = {}
    if s["out"] == "fp8":
        got = w4.w4a16_rmsnorm_fp8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        out["q"], out["scales"] = got[:2]
    else:
        got = w4.w4a16_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        got = got if isinstance(got, tuple) else (got,)
        out["y"] = got[0]
    if s["residual"] is not None:
        out["sum"] = got[-1]
    return out


def run(state):
    return _call(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _e4m3_values():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    vals = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0
                                                  else (1 + m / 8) * 2.0 ** (e - 7))
        vals.append(-v if c & 128 else v)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _decode(q):
    return _e4m3_values()[q.view(torch.uint8).to(torch.int32)]


def _round_e4m3(v):
    """v to the nearest e4m3 value, ties to an even last bit (|v| <= 448)."""
    exponent = torch.frexp(v)[1] - 1  # v = 1.f * 2^exponent
    step = torch.exp2(exponent.clamp(min=-6).double() - 3)  # of subnormals too: 2^-9
    return torch.round(v / step) * step


def _exact_rows8(v):
    M, N = v.shape
    q = torch.empty((M, N), dtype=torch.float64, device=v.device)
    scales = torch.empty((M, -(-N // GROUP)), dtype=torch.float64, device=v.device)
    for g in range(scales.shape[1]):
        part = v[:, g * GROUP:(g + 1) * GROUP]
        fine = torch.isfinite(part)
        top = torch.where(fine, part.abs(), 0.0).amax(1)
        scales[:, g] = torch.maximum(top, torch.full_like(top, FLOOR)) / E4M3_MAX
        r = _round_e4m3(torch.where(fine, part, 0.0) / scales[:, g:g + 1])
        q[:, g * GROUP:(g + 1) * GROUP] = torch.where(fine, r, math.nan)
    return q, scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x, w = _decode(s["x"]), _decode(s["w"])
        y = torch.zeros((M, N), dtype=torch.float64, device="cuda")
        x64, w64 = s["x_scales"].double(), s["w_scales"].double()
        column = torch.arange(K, device="cuda") // GROUP
        x *= x64[:, column]
        for n0 in range(0, N, GROUP):
            y[:, n0:n0 + GROUP] = x @ (w[n0:n0 + GROUP] * w64[n0 // GROUP][column]).t()
        if s["residual"] is not None:
            y += s["residual"].double()
        return {"y": y}
    v = s["x"].double()
    out = {}
    if case["op"] == "quant":
        if case["silu"]:
            gate, up = v.split(case["N"], dim=1)
            v = gate * torch.sigmoid(gate) * up
        out["q"], out["scales"] = _exact_rows8(v)
        return out
    if s["residual"] is not None:
        v = v + s["residual"].double()
        out["sum"] = v
    v = v / (v.square().sum(1, keepdim=True) / case["N"] + EPS).sqrt() * s["weight"].double()
    if case["out"] == "fp8":
        out["q"], out["scales"] = _exact_rows8(v)
    else:
        out["y"] = v
    return out
