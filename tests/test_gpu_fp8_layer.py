"""The 8-bit layer of examples/fp8_layer.py: its steps run together on one
residual stream, each kernel's output compared with the definition (binary64) on
the inputs that the kernels before it left; the captured step gives the same bits;
the layer is close to 32-bit arithmetic on the unquantised weights.

Tolerances: test_gpu_fp8_linear's bound for the linears, and its derivation; the
layer against unquantised weights: an element of a row or weight is off by at most
2^-4 of itself, uniformly over that range on average 2^-4 / sqrt(3) / 2 in root mean
square or less, the two operands of a product independently: sqrt(2) x 1.8% for
each linear, which four linears in a row at most add up: 0.11.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8_linear import bound

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "fp8_layer", os.path.join(ROOT, "examples", "fp8_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.w4.w4a16_init(0, 64 << 20)
    return m


def check(y, rows, weights, residual):
    want, A = ref.linear(rows[0].cpu(), rows[1].cpu(), weights[0].cpu(), weights[1].cpu(),
                         None if residual is None else residual.cpu())
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= bound(want, A, rows[0].shape[1], y.dtype)), float(err.max())


@pytest.mark.parametrize("M", [1, 7, 64, 100, 300])
def test_layer_step_by_step(example, M):
    w4 = example.w4
    hidden, heads, qkv, inter = 640, 768, 1024, 1152
    layer, w = example.random_layer(3, hidden, heads, qkv, inter, max_tokens=320)

    def attention(t):
        return t[:, :heads].contiguous()

    h0 = torch.randn((M, hidden), device="cuda").to(torch.bfloat16)
    h = h0.clone()
    out = layer.step(h, attention)
    assert out.data_ptr() == h.data_ptr()
    # the same steps again, one by one
    q, s = w4.w4a16_rmsnorm_fp8(h0, w["norm1"])
    y = w4.w4a16_fp8_linear(q, s, *layer.wqkv)
    check(y, (q, s), layer.wqkv, None)
    qa = w4.w4a16_fp8_quant(attention(y))
    h1 = w4.w4a16_fp8_linear(*qa, *layer.wo, epilogue=w4.EPILOGUE_RESIDUAL, residual=h0)
    check(h1, qa, layer.wo, h0)
    q2 = w4.w4a16_rmsnorm_fp8(h1, w["norm2"])
    gate_up = w4.w4a16_fp8_linear(*q2, *layer.wgate_up)
    check(gate_up, q2, layer.wgate_up, None)
    qi = w4.w4a16_fp8_quant(gate_up, epilogue=w4.EPILOGUE_SILU_MUL)
    h2 = w4.w4a16_fp8_linear(*qi, *layer.wdown, epilogue=w4.EPILOGUE_RESIDUAL, residual=h1)
    check(h2, qi, layer.wdown, h1)
    assert torch.equal(h, h2)
    # captured
    h = h0.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.step(h, attention)
    h.copy_(h0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, h2)
    # against the unquantised layer
    want = example.reference_step(w, h0, attention)
    off = float((h.float() - want).norm() / (want - h0.float()).norm())
    assert off <= 0.11, off
    assert w4.w4a16_device_status() == 0


def test_new_outputs_on_another_stream_are_its_own_memory(example):
    # memory that the current stream has just freed may still be in use there: a call on
    # another stream has to take its outputs from elsewhere, and to leave them whole for
    # the current stream after they are freed
    w4 = example.w4
    s = torch.cuda.Stream()
    M, H = 256, 2048
    x = torch.randn((M, H), device="cuda").to(torch.bfloat16)
    weight = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones((H, H), device="cuda").to(torch.float8_e4m3fn)
    ws = torch.ones((H // 128, H // 128), device="cuda")
    q, sc = w4.w4a16_fp8_quant(x)
    torch.cuda.synchronize()
    calls = [lambda: w4.w4a16_fp8_linear(q, sc, w, ws, stream=s),
             lambda: w4.w4a16_rmsnorm(x, weight, stream=s),
             lambda: w4.w4a16_rmsnorm(x, weight, residual=x, stream=s),
             lambda: w4.w4a16_rmsnorm_fp8(x, weight, stream=s),
             lambda: w4.w4a16_fp8_quant(x, stream=s)]
    for f in calls:
        freed = [torch.empty(n, dtype=torch.uint8, device="cuda")
                 for n in (2 * M * H, 2 * M * H, M * H, M * H, M * H // 32)]
        spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in freed]
        del freed
        out = f()
        for t in out if isinstance(out, tuple) else (out,):
            a, b = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
            assert all(b <= lo or a >= hi for lo, hi in spans)
        s.synchronize()
