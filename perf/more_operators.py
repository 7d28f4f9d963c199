"""What is timed of the products whose weights a row chooses for itself: the choice
of experts from a router's logits, a layer of experts with 8-bit weights for a few
tokens, and the low-rank adapters of many requests beside a shared projection.

  route    ids [T, k]: the k largest of a row's logits, in falling order, equal ones
           by index (NaN counts as -Inf).  p = softmax(row) or 1 / (1 + e^-logit),
           0 where the logit is -Inf; the weights are p of the chosen, divided by
           their sum with `renorm` (0 where that is 0)
  experts  out[t] = sum_j weight[t, j] * down_e(silu(gate_e(x[t])) * up_e(x[t])),
           e = ids[t, j].  Weights in 8 bits: w [E, rows, cols] e4m3 (4 exponent and 3
           mantissa bits) with one fp32 scale per block of 128 x 128, the gate's
           rows before the up projection's; silu(g) = g / (1 + e^-g)
  adapter  y[m] = residual[m] + scale_l * B_l (A_l x[m]), l = ids[m]; a row whose
           id is not in [0, L) has no adapter.  The projection's columns come in
           parts (q, k and v; gate and up), each with R rows of A of its own:
           a [L, parts * R, K], b [L, N, R].  An adapter uses the first ranks[l]
           of R

With ``own`` false, ``run`` computes this with elementary torch operations in
32 bits; with ``own`` true it makes the calls of this package.
"""
import functools
import math

import torch

own = False

BLOCK = 128
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # --- the choice of experts
        # one decoded token, logits as a 16-bit linear leaves them: latency
        dict(name="route t1 e128", op="route", T=1, E=128, k=8, dtype="bf16", score="softmax",
             renorm=True),
        # a ragged batch over a number of experts that fits nothing
        dict(name="route t77 e61 odd", op="route", T=77, E=61, k=5, dtype="f32", score="sigmoid",
             renorm=False),
        # a long prompt's tokens
        dict(name="route t8192 e256", op="route", T=8192, E=256, k=8, dtype="f32",
             score="softmax", renorm=True),
        # --- the layer of experts (128 experts, 8 per token, 2048 -> 2 x 768 -> 2048)
        # one decoded token
        dict(name="experts t1 e128", op="experts", T=1, E=128, k=8, K=2048, I=768, N=2048,
             dtype="bf16"),
        # a verify pass, or eight requests
        dict(name="experts t8 e128", op="experts", T=8, E=128, k=8, K=2048, I=768, N=2048,
             dtype="f16"),
        # few experts that each see several tokens, sizes that are multiples of nothing
        dict(name="experts t37 e10 odd", op="experts", T=37, E=10, k=3, K=1040, I=336, N=1021,
             dtype="f16"),
        # a decode batch in which nearly every expert is used: the weights' bytes
        dict(name="experts t64 e128", op="experts", T=64, E=128, k=8, K=2048, I=768, N=2048,
             dtype="bf16"),
        # --- adapters beside the decode layer's projections
        # one request beside qkv
        dict(name="adapter m1 qkv", op="adapter", M=1, seqs=1, K=5120, parts="6144,1024,1024",
             L=8, R=16, ragged=False, dtype="bf16", residual=True),
        # a ragged batch of short pieces, ranks that differ, odd sizes
        dict(name="adapter m37 odd", op="adapter", M=37, seqs=9, K=1040, parts="1021", L=5, R=24,
             ragged=True, dtype="f16", residual=True),
        # a decode batch of 64 requests over 32 adapters, beside gate+up
        dict(name="adapter m64 gate_up", op="adapter", M=64, seqs=64, K=5120,
             parts="17408,17408", L=32, R=16, ragged=False, dtype="bf16", residual=True),
        # short prompts beside the attention's output projection
        dict(name="adapter m1000 o", op="adapter", M=1000, seqs=12, K=6144, parts="5120", L=4,
             R=64, ragged=True, dtype="bf16", residual=True),
        # a prefill chunk of eight prompts, beside gate+up
        dict(name="adapter m4096 gate_up", op="adapter", M=4096, seqs=8, K=5120,
             parts="17408,17408", L=8, R=64, ragged=False, dtype="bf16", residual=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "adapter", "adapter"])
    if op == "route":
        E = _spread(rng, 4, 512)
        return dict(op=op, T=_spread(rng, 1, 8192 * 256 // max(E, 256)), E=E,
                    k=rng.randint(1, min(E, 16)), dtype=rng.choice(["f32", "f16", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5)
    dtype = rng.choice(["f16", "bf16"])
    if op == "experts":
        while True:
            E, T = _spread(rng, 4, 160), _spread(rng, 1, 64)
            k = rng.randint(1, min(E, 8))
            K, I = 16 * _spread(rng, 16, 448), 16 * _spread(rng, 8, 128)
            if E * K * I <= 128 * 2048 * 768:
                break
        if rng.random() < 0.5:  # half of them in whole blocks, as layers mostly are
            K, I = -(-K // BLOCK) * BLOCK, -(-I // BLOCK) * BLOCK
        if E * K * I > 128 * 2048 * 768:
            I = 256
        return dict(op=op, T=T, E=E, k=k, K=K, I=I, N=K if rng.random() < 0.5 else K - 3,
                    dtype=dtype)
    while True:
        M = _spread(rng, 1, 8192)
        K = 8 * _spread(rng, 32, 2176)
        parts = [_spread(rng, 64, 17408) for _ in range(rng.randint(1, 3))]
        if rng.random() < 0.5:
            parts = [-(-n // BLOCK) * BLOCK for n in parts]
        L, R = _spread(rng, 1, 64), 8 * rng.randint(1, 16)
        N, S = sum(parts), len(parts)
        if (M * N <= 4096 * 34816 and M * L * R * (S * K + N) <= 4096 * 512 * (10240 + 34816)
                and M * R * (S * K + N) <= 4096 * 64 * (10240 + 34816)
                and L * R * (S * K + N) <= 64 * 16 * (10240 + 34816)):
            break
    # tokens of their own requests, or prompts of many
    seqs = M if M <= 256 and rng.random() < 0.7 else rng.randint(1, max(1, min(M, 32)))
    return dict(op=op, M=M, seqs=seqs, K=K, parts=",".join(map(str, parts)), L=L, R=R,
                ragged=rng.random() < 0.5, dtype=dtype, residual=rng.random() < 0.8)


def _parts(case):
    return [int(n) for n in case["parts"].split(",")]


def _chosen(n, picks):
    """Of n, how many are expected among so many even picks."""
    return n * (1.0 - (1.0 - 1.0 / n) ** picks)


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (4 if case["dtype"] == "f32" else 2) + 8 * T * k,
                "flops": 4 * T * E}
    if case["op"] == "experts":
        T, E, k, K, I, N = (case[n] for n in ("T", "E", "k", "K", "I", "N"))
        used = E * (1.0 - (1.0 - k / E) ** T)
        weights = 2 * I * K + N * I
        scales = (-(-2 * I // BLOCK)) * (-(-K // BLOCK)) + (-(-N // BLOCK)) * (-(-I // BLOCK))
        return {"bytes": int(used * (weights + 4 * scales)) + 2 * T * (K + N) + 8 * T * k,
                "flops": 2 * T * k * weights}
    M, K, L, R = case["M"], case["K"], case["L"], case["R"]
    parts = _parts(case)
    N, S = sum(parts), len(parts)
    rank = (R + 8) / 2 if case["ragged"] else R  # an adapter's, on average
    per = rank * (S * K + N)
    return {"bytes": int(2 * _chosen(L, case["seqs"]) * per) + 2 * M * K
            + 2 * M * N * (2 if case["residual"] else 1) + 4 * M,
            "flops": int(2 * M * per)}


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


def _weights8(gen, E, rows, cols):
    """(e4m3 [E, rows, cols], scales [E, ceil(rows/128), ceil(cols/128)]) of weights with a
    standard deviation of about cols^-1/2; a block's largest code is near 448."""
    q = _normal(gen, (E, rows, cols), torch.float32, 112.0).clamp_(-448.0, 448.0)
    scales = torch.rand((E, -(-rows // BLOCK), -(-cols // BLOCK)), generator=gen, device="cuda")
    return q.to(torch.float8_e4m3fn), (0.75 + 0.5 * scales) * (cols ** -0.5 / 112.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "route":
        s["logits"] = _normal(gen, (case["T"], case["E"]), dt, 2.0)
    elif case["op"] == "experts":
        T, E, k, K, I, N = (case[n] for n in ("T", "E", "k", "K", "I", "N"))
        s["x"] = _activations(gen, T, K, dt)
        top = torch.rand((T, E), generator=gen, device="cuda").topk(k, dim=1)
        s["ids"] = top.indices.to(torch.int32)
        s["weights"] = torch.softmax(4.0 * top.values, dim=1)
        s["w1"], s["s1"] = _weights8(gen, E, 2 * I, K)
        s["w2"], s["s2"] = _weights8(gen, E, N, I)
    else:
        M, K, L, R = case["M"], case["K"], case["L"], case["R"]
        parts = _parts(case)
        N = sum(parts)
        s["x"] = _activations(gen, M, K, dt)
        s["a"] = _normal(gen, (L, len(parts) * R, K), dt, K ** -0.5)
        s["b"] = _normal(gen, (L, N, R), dt, 0.3 * R ** -0.5)
        s["scales"] = 0.5 + 1.5 * torch.rand(L, generator=gen, device="cuda")
        s["ranks"] = None
        if case["ragged"]:
            s["ranks"] = 8 * torch.randint(1, R // 8 + 1, (L,), generator=gen, device="cuda",
                                           dtype=torch.int32)
        # rows in pieces of random lengths, each with an adapter; of many, one in eight without
        cuts = torch.rand(M, generator=gen, device="cuda").argsort() < case["seqs"] - 1
        piece = torch.cumsum(cuts, 0) - cuts.to(torch.int64)
        low = 0 if case["seqs"] < 8 else -max(1, L // 7)
        chosen = torch.randint(low, L, (case["seqs"],), generator=gen, device="cuda")
        s["ids"] = chosen.clamp(min=-1)[piece].to(torch.int32)
        s["residual"] = _normal(gen, (M, N), dt, 4.0) if case["residual"] else None
        s["sizes"] = parts
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _whole_weights(w, scales):
    E, rows, cols = w.shape
    s = scales.repeat_interleave(BLOCK, 1)[:, :rows].repeat_interleave(BLOCK, 2)[:, :, :cols]
    return w.float() * s


def _plain_route(s):
    v = s["logits"].float()
    v = torch.where(torch.isnan(v), -math.inf, v)
    top, ids = torch.sort(v, dim=1, descending=True, stable=True)
    top, ids = top[:, :s["k"]], ids[:, :s["k"]]
    if s["score"] == "softmax":
        most = v.amax(1, keepdim=True)

        def part(z):  # the largest is 1, though it may be infinite
            e = torch.where(z == most, 1.0, torch.exp(z - most))
            return torch.where(z == -math.inf, 0.0, e)

        p, total = part(top), part(v).sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-top))
    if s["renorm"]:
        total = p.sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    return {"ids": ids.to(torch.int32), "weights": p}


def _plain_experts(s):
    E, I = s["E"], s["I"]
    x = s["x"].float()
    both = torch.matmul(x, _whole_weights(s["w1"], s["s1"]).transpose(1, 2))  # [E, T, 2I]
    gate = both[:, :, :I]
    h = gate / (1.0 + torch.exp(-gate)) * both[:, :, I:]
    y = torch.matmul(h, _whole_weights(s["w2"], s["s2"]).transpose(1, 2))     # [E, T, N]
    here = s["ids"][:, :, None] == torch.arange(E, device="cuda")             # [T, k, E]
    share = torch.where(here, s["weights"][:, :, None], 0.0).sum(1)           # [T, E]
    out = (share.t()[:, :, None] * y).sum(0)
    return {"out": out.to(s["x"].dtype)}


def _plain_adapter(s):
    M, K = s["x"].shape
    L, R, sizes = s["L"], s["R"], s["sizes"]
    x = s["x"].float()
    t = (x @ s["a"].float().reshape(L * len(sizes) * R, K).t()).view(M, L, len(sizes), R)
    mine = s["ids"][:, None] == torch.arange(L, device="cuda")                # [M, L]
    keep = mine[:, :, None, None]
    if s["ranks"] is not None:
        keep = keep & (torch.arange(R, device="cuda") < s["ranks"][:, None])[:, None]
    t = torch.where(keep, t * s["scales"][:, None, None], 0.0)
    b = s["b"].float().split(sizes, dim=1)
    y = torch.cat([torch.matmul(t[:, :, i].reshape(M, L * R),
                                b[i].transpose(0, 1).reshape(-1, L * R).t())
                   for i in range(len(sizes))], dim=1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["x"].dtype)}


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
    if s["op"] == "route":
        scoring = w4.ROUTE_SOFTMAX if s["score"] == "softmax" else w4.ROUTE_SIGMOID
        ids, weights = w4.w4a16_moe_route(s["logits"], s["k"], scoring=scoring,
                                          renormalize=s["renorm"])
        return {"ids": ids, "weights": weights}
    if s["op"] == "experts":
        return {"out": w4.w4a16_fp8_moe_mlp(s["x"], s["ids"], s["weights"], s["w1"], s["s1"],
                                            s["w2"], s["s2"])}
    return {"y": w4.w4a16_lora(s["x"], s["a"], s["b"], s["scales"], s["ids"], parts=s["sizes"],
                               ranks=s["ranks"], residual=s["residual"])}


def run(state):
    if own:
        return _call(state)
    return {"route": _plain_route, "experts": _plain_experts,
            "adapter": _plain_adapter}[state["op"]](state)


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


def _exact_weights(w, scales):
    """One expert's weights [rows, cols] in 64 bits."""
    rows, cols = w.shape
    v = _e4m3_values()[w.view(torch.uint8).to(torch.int32)]
    r, c = torch.arange(rows, device="cuda") // BLOCK, torch.arange(cols, device="cuda") // BLOCK
    return v * scales.double()[r[:, None], c[None, :]]


def _exact_route(s):
    z = s["logits"].double().cpu().tolist()
    k, ids, weights = s["k"], [], []
    for row in z:
        row = [-math.inf if math.isnan(v) else v for v in row]
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        if s["score"] == "softmax":
            top = max(row)
            e = [0.0 if v == -math.inf else 1.0 if v == top else math.exp(v - top) for v in row]
            total = math.fsum(e)
            p = [e[i] / total if total > 0 else 0.0 for i in order]
        else:
            p = [0.0 if row[i] == -math.inf else 1.0 / (1.0 + math.exp(-row[i])) for i in order]
        if s["renorm"]:
            total = math.fsum(p)
            p = [v / total if total > 0 else 0.0 for v in p]
        ids.append(order)
        weights.append(p)
    return {"ids": torch.tensor(ids, dtype=torch.int32, device="cuda"),
            "weights": torch.tensor(weights, dtype=torch.float64, device="cuda")}


def _exact_experts(s):
    x, out = s["x"].double(), torch.zeros((s["T"], s["N"]), dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        token, choice = torch.nonzero(s["ids"] == e, as_tuple=True)
        if token.numel() == 0:
            continue
        both = x[token] @ _exact_weights(s["w1"][e], s["s1"][e]).t()
        gate, up = both.split(s["I"], dim=1)
        y = (gate * torch.sigmoid(gate) * up) @ _exact_weights(s["w2"][e], s["s2"][e]).t()
        out.index_add_(0, token, s["weights"][token, choice].double()[:, None] * y)
    return {"out": out}


def _exact_adapter(s):
    M, N, R = s["M"], sum(s["sizes"]), s["R"]
    y = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    ranks = [R] * s["L"] if s["ranks"] is None else s["ranks"].tolist()
    for l in range(s["L"]):
        rows = torch.nonzero(s["ids"] == l).flatten()
        if rows.numel() == 0:
            continue
        x, first = s["x"][rows].double(), 0
        for i, n in enumerate(s["sizes"]):
            a = s["a"][l, i * R:i * R + ranks[l]].double()
            b = s["b"][l, first:first + n, :ranks[l]].double()
            y[rows, first:first + n] = float(s["scales"][l]) * ((x @ a.t()) @ b.t())
            first += n
    if s["residual"] is not None:
        y += s["residual"].double()
    return {"y": y}


def exact(case, seed):
    return {"route": _exact_route, "experts": _exact_experts,
            "adapter": _exact_adapter}[case["op"]](prepare(case, seed))
