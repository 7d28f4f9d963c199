"""The 8-bit linear of one token with nearly 2^31 weight rows (34 GB): rows at both ends
and on both sides of 2^30, and zeros between, exactly."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def test_nearly_2_to_31_weight_rows():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, 64 << 20)
    N, K = 2 ** 31 - 3, 16
    assert w4.w4a16_fp8_plan_info(1, N, K)["grid"] == w4.lib.w4a16_device_sm_count()
    f8 = torch.float8_e4m3fn
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-4, 5, (1, K), generator=g, device=DEV).float().to(f8)
    xs = torch.full((1, 1), 0.5, device=DEV)
    w = torch.zeros((N, K), dtype=torch.uint8, device=DEV).view(f8)
    ws = torch.full((-(-N // 128), 1), 2.0, device=DEV)
    spans = [(0, 384), (2 ** 30 - 256, 2 ** 30 + 256), (N // 128 * 128 - 256, N)]
    for a, b in spans:
        w[a:b] = torch.randint(-4, 5, (b - a, K), generator=g, device=DEV).float().to(f8)
        ws[a // 128:-(-b // 128)] = torch.rand((-(-b // 128) - a // 128, 1), generator=g,
                                               device=DEV).round() + 0.25
    y = torch.full((1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    w4.w4a16_fp8_linear(x, xs, w, ws, y=y)
    for a, b in spans:
        part = w4.w4a16_fp8_linear(x, xs, w[a:b], ws[a // 128:-(-b // 128)])
        assert part.abs().sum() > 0 and torch.equal(y[:, a:b], part)
    ends = [0] + [v for s in spans for v in s]
    for a, b in zip(ends[::2], ends[1::2]):
        for i in range(a, b, 1 << 28):
            assert (y[:, i:min(b, i + (1 << 28))] == 0).all()
    assert w4.w4a16_device_status() == 0
    del w, y, ws
    torch.cuda.empty_cache()
