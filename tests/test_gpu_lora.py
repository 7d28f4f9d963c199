"""The low-rank adapters of many requests (w4a16_lora) against their definition in
binary64: one row to thousands, tall and low tiles and batches that mix them, parts, ranks
that differ, rows without an adapter, odd sizes and addresses, in place, guards, streams,
graphs, beside each of the projections.  The tolerance is derived in routed_reference.py.
"""
import numpy as np
import pytest
import torch

import fp8_reference
import routed_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def w4():
    import __graft_entry__
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    w4.w4a16_init(0, 64 << 20)
    return w4


def on(ops, kw):
    return [t.to(DEV) for t in ops], {n: v.to(DEV) if isinstance(v, torch.Tensor) else v
                                      for n, v in kw.items()}


def check(y, ops, kw, dtype):
    want, bound = ref.adapters(*ops, kw["parts"], kw["ranks"], kw["residual"], dtype)
    got = ref.f64(y)
    assert got.shape == want.shape
    err = np.abs(got - want)
    bad = np.argwhere(~(err <= bound))
    assert bad.size == 0, (len(bad), bad[:3].tolist(), float(np.nanmax(err / (bound + 1e-30))))


def run(w4, ops, kw):
    o, k = on(ops, kw)
    return w4.w4a16_lora(*o, **k)


SHAPES = [  # M, K, parts, L, R
    (1, 8, (1,), 1, 8), (1, 512, (256, 64, 64), 4, 16), (1, 5120, (1024,), 2, 64),
    (2, 72, (9, 7), 3, 8), (3, 640, (130,), 2, 24), (7, 1040, (1021,), 5, 24),
    (16, 256, (384, 384), 2, 32), (17, 264, (96, 40, 8, 16), 1, 40), (33, 1024, (520,), 40, 16),
    (37, 1040, (1021,), 5, 56), (64, 2048, (768, 768), 32, 16), (100, 384, (257,), 1, 128),
    (129, 136, (200,), 1, 72), (145, 520, (136, 264), 2, 8), (256, 1000, (512,), 3, 64),
    (200, 256, (136,), 2, 128), (300, 640, (640, 128, 128), 4, 48), (1000, 256, (320,), 6, 64), (1025, 64, (72,), 1024, 8),
    (4100, 128, (136,), 3, 16),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,parts,L,R", SHAPES)
def test_matches_definition(w4, M, K, parts, L, R, dtype):
    for ranks, residual in ((False, True), (True, False)):
        ops, kw = ref.make_adapters(M + K, M, K, parts, L, R, dtype, ranks=ranks, residual=residual)
        check(run(w4, ops, kw), ops, kw, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("counts", [(16,), (17,), (128,), (129,), (143,), (144,), (145,),
                                    (1, 16, 17, 127, 0, 128, 300, 3), (0, 0, 5)])
def test_tiles_of_every_height(w4, counts, dtype):
    L, M = len(counts), sum(counts)
    ids = torch.cat([torch.full((n,), l, dtype=torch.int32) for l, n in enumerate(counts)])
    ids = ids[torch.randperm(M, generator=torch.Generator().manual_seed(1))]
    ops, kw = ref.make_adapters(5, M, 328, (72, 56), L, 24, dtype, ids=ids, ranks=True)
    check(run(w4, ops, kw), ops, kw, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [9, 200])
def test_rows_without_an_adapter(w4, M, dtype):
    ops, kw = ref.make_adapters(2, M, 256, (48, 32), 3, 16, dtype)
    ids = ops[4]
    ids[::2] = torch.tensor([-1, -7, 3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[
        torch.arange((M + 1) // 2) % 5]
    kw["residual"][0, :3] = torch.tensor([-0.0, float("nan"), float("inf")])
    plain = (ids < 0) | (ids >= 3)
    y = run(w4, ops, kw)
    bits = torch.int16
    assert torch.equal(y.cpu()[plain].view(bits), kw["residual"][plain].view(bits))
    kw["residual"][0, :3] = 0
    check(run(w4, ops, kw), ops, kw, dtype)
    # nobody has one; all ranks 0; no residual either
    none = torch.full_like(ids, -1)
    y = run(w4, (*ops[:4], none), kw)
    assert torch.equal(y.cpu().view(bits), kw["residual"].view(bits))
    kw["ranks"] = torch.tensor([0, -3, 0], dtype=torch.int32)
    y = run(w4, ops, kw)
    assert torch.equal(y.cpu().view(bits), kw["residual"].view(bits))
    kw["residual"] = None
    assert bool((run(w4, ops, kw) == 0).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [5, 150])
def test_nothing_beyond_a_rank_is_used(w4, M, dtype):
    ops, kw = ref.make_adapters(4, M, 200, (40, 88), 4, 32, dtype,
                                ids=torch.arange(M, dtype=torch.int32) % 4)
    kw["ranks"] = torch.tensor([5, 16, 31, 9], dtype=torch.int32)
    nan = float("nan")
    for l, r in enumerate(kw["ranks"].tolist()):
        ops[2][l, :, r:] = nan
        for p in range(2):
            ops[1][l, p * 32 + r:(p + 1) * 32] = nan
    check(run(w4, ops, kw), ops, kw, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M", [6, 140])
def test_values_far_from_one(w4, M, dtype):
    # A x beyond the 16-bit type's range on either side, and rows that are not finite
    ops, kw = ref.make_adapters(6, M, 256, (64, 24), 2, 16, dtype,
                                ids=torch.arange(M, dtype=torch.int32) % 2, residual=False)
    ops[0][0] *= 2.0 ** 12
    ops[1][0] *= 2.0 ** 9
    ops[2][0] *= 2.0 ** -12
    ops[3][0] *= 2.0 ** -12
    ops[0][1] *= 2.0 ** -10
    ops[1][1] *= 2.0 ** -6
    check(run(w4, ops, kw), ops, kw, dtype)
    ops[0][2, 3], ops[0][3, 100] = float("inf"), float("nan")
    y = ref.f64(run(w4, ops, kw))
    assert not np.isfinite(y[2]).any() and np.isnan(y[3]).all()
    rows = [m for m in range(M) if m not in (2, 3)]
    ops[0][2:4] = 0
    want, bound = ref.adapters(*ops, kw["parts"], None, None, dtype)
    assert np.all((np.abs(y - want) <= bound)[rows])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,parts", [(11, (64, 32)), (11, (63, 32)), (170, (64, 32)),
                                     (170, (61, 35))])
def test_in_place_guards_and_odd_addresses(w4, M, parts, dtype):
    N = sum(parts)
    ops, kw = ref.make_adapters(7, M, 256, parts, 3, 16, dtype)
    want = run(w4, ops, kw)
    o, k = on(ops, kw)
    got = w4.w4a16_lora(*o, **{**k, "y": k["residual"]})
    assert got.data_ptr() == k["residual"].data_ptr() and torch.equal(got, want)
    o, k = on(ops, kw)
    for shift in (0, 1):  # an address that 16-byte accesses do not fit
        room = torch.full((M * N + 2 * N + shift,), 5.0, dtype=dtype, device=DEV)
        y = room[N + shift:N + shift + M * N].view(M, N)
        assert torch.equal(w4.w4a16_lora(*o, **k, y=y), want)
        assert bool((room[:N + shift] == 5).all()) and bool((room[N + shift + M * N:] == 5).all())
    res = torch.empty(M * N + 1, dtype=dtype, device=DEV)[1:].view(M, N).copy_(k["residual"])
    assert torch.equal(w4.w4a16_lora(*o, **{**k, "residual": res}), want)
    # an empty batch
    k["residual"] = k["residual"][:0]
    assert w4.w4a16_lora(o[0][:0], *o[1:4], o[4][:0], **k).shape == (0, N)


def test_same_bits_every_time_on_any_stream_and_in_graphs(w4):
    sets = [on(*ref.make_adapters(1, 300, 1024, (256, 256), 7, 32, BF16)),
            on(*ref.make_adapters(2, 40, 1024, (256, 256), 7, 32, BF16))]
    want = [w4.w4a16_lora(*o, **k) for o, k in sets]
    for _ in range(10):
        for (o, k), w in zip(sets, want):
            assert torch.equal(w4.w4a16_lora(*o, **k), w)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):  # two at a time
        got += [w4.w4a16_lora(*o, **k, stream=s) for (o, k), s in zip(sets, streams)]
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    graphs, outs = [], []
    for o, k in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(w4.w4a16_lora(*o, **k))
        graphs.append(graph)
    for s, graph in zip(streams, graphs):  # two replays at once
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(outs, want))
    # other rows and adapters under the same graph
    o, k = sets[0]
    n, kn = ref.make_adapters(9, 300, 1024, (256, 256), 7, 32, BF16)
    for to, new in zip(o, n):
        to.copy_(new)
    k["residual"].copy_(kn["residual"])
    graphs[0].replay()
    check(outs[0], n, kn, BF16)


def test_rows_do_not_depend_on_their_place(w4):
    # the same rows in another order: the same bits, whatever tiles they fall in (one adapter
    # has a tall tile and a few rows more)
    ids = torch.tensor([0] * 140 + [1] * 100 + [2] * 12 + [-1] * 8, dtype=torch.int32)
    ops, kw = ref.make_adapters(3, 260, 2048, (128,), 4, 16, BF16, ids=ids)
    o, k = on(ops, kw)
    want = w4.w4a16_lora(*o, **k)
    for seed in range(10):
        perm = torch.randperm(260, generator=torch.Generator().manual_seed(seed)).to(DEV)
        got = w4.w4a16_lora(o[0][perm], *o[1:4], o[4][perm], parts=kw["parts"],
                            residual=k["residual"][perm])
        assert torch.equal(got, want[perm])


@pytest.mark.parametrize("M", [3, 70])
def test_beside_the_projections(w4, M):
    """A fused qkv projection of 16-bit rows and an 8-bit one, each followed by the rows'
    adapters in place, as a decoder layer calls them, on a captured stream."""
    K, parts, L, R = 256, (256, 128, 128), 3, 16
    N = sum(parts)
    ops, kw = ref.make_adapters(8, M, K, parts, L, R, BF16)
    (x, a, b, scales, ids), _ = on(ops, kw)
    w = (torch.randn((N, K), generator=torch.Generator().manual_seed(3)) * K ** -0.5).to(BF16).to(DEV)
    f8, ws = (w.float() * 64).to(torch.float8_e4m3fn), torch.full((N // 128, K // 128), 2.0 ** -6,
                                                                 device=DEV)
    q, qs = w4.w4a16_fp8_quant(x)

    def layer():
        y = w4.w4a16_dense_linear(x, w)
        base = y.clone()
        w4.w4a16_lora(x, a, b, scales, ids, parts=parts, residual=y, y=y)
        y8 = w4.w4a16_fp8_linear(q, qs, f8, ws)
        z = w4.w4a16_lora(x, a, b, scales, ids, parts=parts, residual=y8)
        return base, y, y8, z

    eager = layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(e, c) for e, c in zip(eager, captured))
    base, y, y8, z = eager
    for res, out in ((base, y), (y8, z)):
        check(out, ops, dict(parts=parts, ranks=None, residual=res.cpu()), BF16)
    want = fp8_reference.linear(q.cpu(), qs.cpu(), f8.cpu(), ws.cpu())[0]
    assert np.all(np.abs(ref.f64(y8) - want) <= 2.0 ** -7 * np.abs(want).max())
    assert w4.w4a16_device_status() == 0


def test_outputs_beyond_32_bits(w4):
    # 65535 rows of 34816: 4.6 GB of y, elements past 2^31; rows of all parts, compared where
    # they lie at both ends and around the limit
    M, K, parts, L, R = 65535, 64, (17408, 17408), 2, 8
    rows = [0, 1, 61679, 61680, 65533, 65534]  # 2^31 / 34816 = 61680.9
    ops, kw = ref.make_adapters(10, len(rows), K, parts, L, R, BF16,
                                ids=torch.tensor([0, 1, 0, 1, -1, 1], dtype=torch.int32))
    x = torch.randn((M, K), device=DEV).to(BF16)
    ids = torch.arange(M, dtype=torch.int32, device=DEV) % 3 - 1
    y = torch.zeros((M, 2 * 17408), dtype=BF16, device=DEV)
    x[rows], ids[rows], y[rows] = ops[0].to(DEV), ops[4].to(DEV), kw["residual"].to(DEV)
    w4.w4a16_lora(x, ops[1].to(DEV), ops[2].to(DEV), ops[3].to(DEV), ids, parts=parts, residual=y,
                  y=y)
    check(y[rows], ops, kw, BF16)
    assert w4.w4a16_device_status() == 0
