"""The linears of a decoder layer in 8 bits, around an attention of the caller's:

    q8      = norm(h)                     w4a16_rmsnorm_fp8
    qkv     = q8 @ Wqkv^T                 w4a16_fp8_linear
    a       = attention(qkv)              the caller's (here: a stand-in that takes columns)
    h      += quant(a) @ Wo^T             w4a16_fp8_quant, w4a16_fp8_linear with the residual
    q8      = norm(h)                     w4a16_rmsnorm_fp8
    gate_up = q8 @ Wgu^T                  w4a16_fp8_linear
    h      += quant(silu(gate) up) @ Wd^T w4a16_fp8_quant (silu-and-mul), w4a16_fp8_linear

Every activation that enters a linear is 8 bits with a scale per 128 elements,
every weight 8 bits with a scale per 128 x 128 block; the residual stream h, qkv
and gate_up are 16 bits.  The layer allocates its buffers once, so that a step
can be captured into a CUDA graph.

    python examples/fp8_layer.py --tokens 8 --layers 8

prints the time per layer and the layer's error against 32-bit torch arithmetic on
the weights before they were quantised.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_int4_w4a16_gb300 as w4  # noqa: E402

BLOCK = 128
FP8 = torch.float8_e4m3fn


def quantise_weight(w: torch.Tensor):
    """[N, K] -> (e4m3 [N, K], scales [ceil(N/128), ceil(K/128)]), at load time.
    (A checkpoint that comes in this form needs no such step.)"""
    N, K = w.shape
    b = torch.nn.functional.pad(w.float(), (0, -K % BLOCK, 0, -N % BLOCK))
    b = b.view(b.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    scales = b.abs().amax((1, 3)).clamp(min=2.0 ** -100) / 448.0
    q = (b / scales[:, None, :, None]).reshape(b.shape[0] * BLOCK, -1)[:N, :K]
    return q.to(FP8).contiguous(), scales


class Fp8Layer:
    """One layer's weights and the buffers of a step of up to max_tokens tokens."""

    def __init__(self, norm1, wqkv, wo, norm2, wgate_up, wdown, max_tokens: int, eps=1e-6):
        self.norm1, self.norm2, self.eps = norm1, norm2, eps
        self.wqkv, self.wo = quantise_weight(wqkv), quantise_weight(wo)
        self.wgate_up, self.wdown = quantise_weight(wgate_up), quantise_weight(wdown)
        dev, dt, M = norm1.device, norm1.dtype, max_tokens
        self.hidden, self.heads, self.inter = wqkv.shape[1], wo.shape[1], wdown.shape[1]

        def rows(n):
            return (torch.empty((M, n), dtype=FP8, device=dev),
                    torch.empty((M, -(-n // BLOCK)), dtype=torch.float32, device=dev))

        self.q_hidden, self.q_heads = rows(self.hidden), rows(self.heads)
        self.q_inter = rows(self.inter)
        self.qkv = torch.empty((M, wqkv.shape[0]), dtype=dt, device=dev)
        self.gate_up = torch.empty((M, wgate_up.shape[0]), dtype=dt, device=dev)

    def step(self, h: torch.Tensor, attention) -> torch.Tensor:
        """One layer over the residual stream h [M, hidden], which it updates in place."""
        M, dt = h.shape[0], h.dtype
        q, s = (t[:M] for t in self.q_hidden)
        w4.w4a16_rmsnorm_fp8(h, self.norm1, eps=self.eps, q=q, scales=s)
        qkv = w4.w4a16_fp8_linear(q, s, *self.wqkv, dtype=dt, y=self.qkv[:M])
        a = attention(qkv)
        qa, sa = (t[:M] for t in self.q_heads)
        w4.w4a16_fp8_quant(a, q=qa, scales=sa)
        w4.w4a16_fp8_linear(qa, sa, *self.wo, dtype=dt, epilogue=w4.EPILOGUE_RESIDUAL, residual=h,
                            y=h)
        w4.w4a16_rmsnorm_fp8(h, self.norm2, eps=self.eps, q=q, scales=s)
        gate_up = w4.w4a16_fp8_linear(q, s, *self.wgate_up, dtype=dt, y=self.gate_up[:M])
        qi, si = (t[:M] for t in self.q_inter)
        w4.w4a16_fp8_quant(gate_up, epilogue=w4.EPILOGUE_SILU_MUL, q=qi, scales=si)
        return w4.w4a16_fp8_linear(qi, si, *self.wdown, dtype=dt, epilogue=w4.EPILOGUE_RESIDUAL,
                                   residual=h, y=h)


def random_layer(seed, hidden, heads, qkv, inter, max_tokens, dt=torch.bfloat16, device="cuda"):
    """(Fp8Layer, its weights before quantisation) of a seeded random layer."""
    g = torch.Generator(device=device).manual_seed(seed)

    def weight(n, k):
        return torch.randn((n, k), generator=g, device=device).mul_(k ** -0.5).to(dt)

    def norm():
        return (1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(dt)

    w = dict(norm1=norm(), wqkv=weight(qkv, hidden), wo=weight(hidden, heads), norm2=norm(),
             wgate_up=weight(2 * inter, hidden), wdown=weight(hidden, inter))
    return Fp8Layer(**w, max_tokens=max_tokens), w


def reference_step(w, h, attention, eps=1e-6):
    """The same layer in 32-bit torch arithmetic on unquantised weights."""
    def norm(v, weight):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * weight.float()

    h = h.float()
    qkv = norm(h, w["norm1"]) @ w["wqkv"].float().t()
    h = h + attention(qkv) @ w["wo"].float().t()
    gate, up = (norm(h, w["norm2"]) @ w["wgate_up"].float().t()).chunk(2, -1)
    return h + (torch.nn.functional.silu(gate) * up) @ w["wdown"].float().t()


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--layers", type=int, default=8)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    w4.w4a16_init(0)
    hidden, heads, qkv, inter = 5120, 6144, 8192, 17408  # the decode layer's linears
    layers = [random_layer(i, hidden, heads, qkv, inter, a.tokens) for i in range(a.layers)]

    def attention(t):  # stands in for the caller's: a contiguous [M, heads]
        return t[:, :heads].contiguous()

    h0 = torch.randn((a.tokens, hidden), device="cuda").to(torch.bfloat16)
    h = h0.clone()
    layers[0][0].step(h, attention)
    want = reference_step(layers[0][1], h0, attention)
    added = (want - h0.float()).norm()
    print(f"layer 0: |h - reference| / |what the layer adds| = "
          f"{float((h.float() - want).norm() / added):.4f}")
    for _, w in layers:
        w.clear()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for layer, _ in layers:
            layer.step(h, attention)
    graph.replay()
    begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert w4.w4a16_device_status() == 0
    us = begin.elapsed_time(end) * 1e3 / a.steps / a.layers
    weights = qkv * hidden + hidden * heads + 3 * hidden * inter
    print(f"{a.tokens} tokens: {us:.1f} us per layer ({weights / us / 1e3:.0f} GB/s of weights, "
          f"{2 * a.tokens * weights / us / 1e6:.1f} TFLOP/s)")


if __name__ == "__main__":
    main()
