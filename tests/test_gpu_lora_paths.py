"""The low-rank adapters (w4a16_lora) on every path of theirs, each named by the plan that the
library gives for the sizes: the kinds of the first product with the rows grouped in every CTA
and before, more than one block of 128 rows of A, and outputs whose columns fit no 16 bytes in
tall and low tiles of every rank's kernel.  The tolerance is derived in routed_reference.py.
"""
import pytest
import torch

import routed_reference as ref
from test_gpu_lora import check, run

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, 64 << 20)
    return w4


def test_a_cluster_for_every_unit_of_few_rows(w4):
    # the most tiles of 16 rows that so many rows of so many adapters can make
    for M, L, R, parts in ((127, 1, 16, 1), (100, 1, 16, 1), (128, 2, 16, 3), (17, 1, 8, 1),
                           (128, 1, 32, 2), (50, 40, 16, 1), (1, 1024, 8, 1), (113, 7, 16, 4)):
        used = min(M, L)
        tiles = max(sum(-(-n // 16) for n in counts)
                    for counts in ([M - used + 1] + [1] * (used - 1),
                                   [M // used + (i < M % used) for i in range(used)]))
        p = w4.w4a16_lora_plan_info(M, L, R, parts)
        assert p["kind"] == 0 and p["kernels"] == 2
        assert p["clusters"] >= min(tiles * -(-parts * R // 32), 38)


def grouped(M, L, seed):
    """Ids with tall and low adapters: half of the rows on the first, the others spread."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    ids[torch.rand(M, generator=g) < 0.5] = 0
    if L > 2:  # a low tile of 11 rows
        ids[ids == L - 1] = L - 2
        ids[torch.randperm(M, generator=g)[:11]] = L - 1
    return ids


CASES = [  # M, K, parts, L, R, kind (None: by how many clusters the device holds), kernels
    (130, 136, (61, 35), 3, 8, 1, 2), (257, 264, (1021,), 4, 24, 1, 2),
    (300, 200, (257, 130, 9), 4, 40, 1, 2), (700, 328, (61, 35), 5, 64, 1, 2),
    (1000, 256, (129,), 3, 128, 1, 2), (1024, 128, (33, 31), 2, 72, None, 2),
    # the rows grouped in every CTA, more tall units than clusters that run at once
    (1000, 256, (72, 56, 40, 24), 5, 128, 2, 2), (900, 264, (61, 35, 127, 1), 4, 128, 2, 2),
    (1024, 72, (130, 64, 3), 3, 128, 2, 2),
    # grouped before
    (1025, 136, (61, 35), 4, 16, 1, 3), (1100, 128, (1021,), 30, 24, 1, 3),
    (4097, 64, (72, 56, 40), 6, 64, 2, 3), (4200, 72, (35, 61), 5, 128, 2, 3),
    (2300, 64, (255,), 3, 48, None, 3),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,parts,L,R,kind,kernels", CASES)
def test_every_path(w4, M, K, parts, L, R, kind, kernels, dtype):
    p = w4.w4a16_lora_plan_info(M, L, R, len(parts))
    assert p["kind"] == kind or kind is None
    assert p["kernels"] == kernels
    for ranks, residual in ((False, True), (True, False)):
        ops, kw = ref.make_adapters(M + R, M, K, parts, L, R, dtype, ids=grouped(M, L, M),
                                    ranks=ranks, residual=residual)
        y = run(w4, ops, kw)
        check(y, ops, kw, dtype)
        assert torch.equal(run(w4, ops, kw), y)
        assert w4.w4a16_device_status() == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("R", [8, 24, 64, 128])
@pytest.mark.parametrize("M", [3, 16, 100])
def test_few_rows_of_every_rank(w4, M, R, dtype):
    for parts in ((61, 35), (64, 40), (1, 1, 1021)):
        ops, kw = ref.make_adapters(M * R, M, 264, parts, 3, R, dtype, ranks=True)
        y = run(w4, ops, kw)
        check(y, ops, kw, dtype)
        assert w4.w4a16_device_status() == 0


@pytest.mark.parametrize("M", [150, 1200])
def test_between_kernels_that_take_all_tensor_memory(w4, M):
    """Tall tiles right after and before the 8-bit linear, whose kernels take all of an SM's
    tensor memory, and with kernels between them that let the next one start at once."""
    K, N, L, R = 256, 512, 3, 64
    ops, kw = ref.make_adapters(M, M, K, (256, 256), L, R, BF16, ids=grouped(M, L, 3))
    x, a, b, scales, ids = [t.cuda() for t in ops]
    g = torch.Generator().manual_seed(1)
    w = (torch.randn((N, K), generator=g) * 4).to(torch.float8_e4m3fn).cuda()
    ws = torch.full((N // 128, K // 128), 2.0 ** -6, device="cuda")
    q, qs = w4.w4a16_fp8_quant(x)
    logits = torch.randn((M, 64), generator=g).cuda()

    def layer():
        outs = []
        for _ in range(3):
            y = w4.w4a16_fp8_linear(q, qs, w, ws)
            outs.append(w4.w4a16_lora(x, a, b, scales, ids, parts=[256, 256], residual=y))
            z = w4.w4a16_fp8_linear(q, qs, w, ws)
            outs.extend(w4.w4a16_moe_route(logits, 4))
            outs.append(w4.w4a16_lora(x, a, b, scales, ids, parts=[256, 256], residual=z))
        return y, outs

    y, eager = layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, captured = layer()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for i, (e, c) in enumerate(zip(eager, captured)):
        assert torch.equal(e, c) and torch.equal(e, eager[i % 4])
    check(eager[0], ops, dict(parts=[256, 256], ranks=None, residual=y.cpu()), BF16)
    assert torch.equal(eager[0], eager[3])
    assert w4.w4a16_device_status() == 0
