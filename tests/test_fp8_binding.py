"""The binding of the 8-bit layer's calls: what it does on a torch without the functions
that are not part of torch's interface, and its refusal of operands on different devices.
"""
import os
import subprocess
import sys

import pytest
import torch

import __graft_entry__

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# run in a process of its own, before the package is imported
WITHOUT = """
import torch
torch.cuda.is_available()
del torch._C._dynamo.guards._empty_strided_cuda
del torch._C._cuda_getCurrentRawStream
own = torch._C._cuda_getDevice
del torch._C._cuda_getDevice
import weight_only_int4_w4a16_gb300 as w4
from weight_only_int4_w4a16_gb300 import binding
assert binding._empty_cuda is None and binding._current_device is torch.cuda.current_device
torch._C._cuda_getDevice = own  # torch's interface needs it too
"""


@pytest.fixture(scope="module")
def binding():
    __graft_entry__.build()
    from weight_only_int4_w4a16_gb300 import binding
    return binding


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_import_without_torch_internals(binding):
    run(WITHOUT)


@pytest.mark.gpu
def test_calls_without_torch_internals(binding):
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((5, 512), generator=g, device="cuda").half()
    want = w4.w4a16_rmsnorm(x, x[0], residual=x) + w4.w4a16_fp8_quant(x)
    y = w4.w4a16_fp8_linear(want[2], want[3], want[2], want[3][:1].contiguous())
    torch.cuda.synchronize()
    run(WITHOUT + """
w4.w4a16_init(0)
g = torch.Generator(device="cuda").manual_seed(3)
x = torch.randn((5, 512), generator=g, device="cuda").half()
for stream in (None, torch.cuda.Stream()):
    torch.cuda.synchronize()
    got = w4.w4a16_rmsnorm(x, x[0], residual=x, stream=stream) + w4.w4a16_fp8_quant(x, stream=stream)
    y = w4.w4a16_fp8_linear(got[2], got[3], got[2], got[3][:1].clone(), stream=stream)
    torch.cuda.synchronize()
    print([float(t.float().sum()) for t in got + (y,)], [t.device for t in got])
    assert all(t.device == x.device for t in got)
    sums = [float(t.double().sum()) for t in (got[0], got[1], got[2].float(), got[3], y)]
    assert sums == SUMS, (sums, SUMS)
""".replace("SUMS", repr([float(t.double().sum())
                          for t in (want[0], want[1], want[2].float(), want[3], y)])))


class On(torch.Tensor):
    """A CPU tensor that says it lives on CUDA device 0 or 1 (a check's double: its address
    reaches no library call here)."""

    @staticmethod
    def make(device, *args, **kw):
        t = torch.zeros(*args, **kw).as_subclass(On)
        t.at = device
        return t

    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at


def test_operands_on_different_devices_are_refused(binding, monkeypatch):
    f8, f16 = torch.float8_e4m3fn, torch.float16
    monkeypatch.setattr(binding, "_current_device", lambda: 0)

    def refuse(*args):
        raise AssertionError("the library was called")

    monkeypatch.setattr(binding, "lib", type("Lib", (), {
        "w4a16_fp8_linear": refuse, "w4a16_rmsnorm": refuse, "w4a16_fp8_quant": refuse}))

    def linear(at):
        a, b, c, d, e, f = at
        return binding.w4a16_fp8_linear(
            On.make(a, (2, 256), dtype=f8), On.make(b, (2, 2)), On.make(c, (64, 256), dtype=f8),
            On.make(d, (1, 2)), binding.EPILOGUE_RESIDUAL, On.make(e, (2, 64), dtype=f16),
            dtype=f16, y=On.make(f, (2, 64), dtype=f16), stream=0)

    monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
    for i, name in enumerate(("x_scales", "w", "w_scales", "residual", "y")):
        at = [0] * 6
        at[i + 1] = 1
        with pytest.raises(ValueError, match=f"{name} must live on cuda:0"):
            linear(at)
    with pytest.raises(ValueError, match="x lives on cuda:1"):
        linear([1] * 6)
    with pytest.raises(AssertionError, match="the library was called"):
        linear([0] * 6)
    x, y = On.make(0, (2, 256), dtype=f16), On.make(1, (2, 256), dtype=f16)
    with pytest.raises(ValueError, match="weight must live on cuda:0"):
        binding.w4a16_rmsnorm(x, On.make(1, (256,), dtype=f16))
    with pytest.raises(ValueError, match="residual must live on cuda:0"):
        binding.w4a16_rmsnorm_fp8(x, On.make(0, (256,), dtype=f16), residual=y)
    with pytest.raises(ValueError, match="x lives on cuda:1"):
        binding.w4a16_fp8_quant(y)
    with pytest.raises(ValueError, match="q must live on cuda:0"):
        binding.w4a16_fp8_quant(x, q=On.make(1, (2, 256), dtype=f8))
