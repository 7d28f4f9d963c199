"""The layer of 8-bit experts (w4a16_fp8_moe_mlp) against its definition in binary64: one
to many tokens, every tile width, sizes that fill no block, choices that are none or
repeated, operands that are not finite, guards, streams, graphs.

Tolerance, per element, with u the unit roundoff of the 16-bit type, A the sum of
magnitudes of a sum's products and G its blocks of 128: a product is exact in fp32; a
block's sum comes from eight instructions of 16 products, every addition off by at most a
unit of the largest term (2^-23, doubled for a truncating adder), scaling and adding the
blocks and the warps' parts rounds at most 8 + G times more: (16 + G) 2^-22 A for gate,
up and down.  h = silu(gate) up moves with gate by at most 1.1 |up|, its exponential and
quotient are off by 2^-20, and it is rounded once (u); the weighted sum rounds twice per
choice (2^-23), out once (u).  2^-24 is the subnormal spacing of fp16.
"""
import numpy as np
import pytest
import torch

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


def dev(ops):
    return [t.to(DEV) for t in ops]


def check(out, want, bound, rows=slice(None)):
    got = ref.f64(out)
    assert got.shape == want.shape
    err = np.abs(got - want)[rows]
    bad = np.argwhere(~(err <= bound[rows]))
    assert bad.size == 0, (len(bad), bad[:3].tolist(), float(np.nanmax(err / bound[rows])))


SHAPES = [  # T, k, E, K, I, N
    (1, 1, 1, 16, 16, 1), (1, 8, 128, 256, 128, 256), (1, 2, 8, 2048, 768, 2048),
    (2, 3, 4, 144, 48, 33), (3, 2, 5, 128, 64, 130), (4, 8, 32, 640, 208, 640),
    (8, 8, 64, 1040, 336, 1021), (9, 4, 16, 272, 112, 400), (13, 2, 3, 512, 144, 257),
    (16, 6, 7, 400, 640, 48), (37, 3, 10, 1040, 336, 1021), (64, 8, 16, 512, 256, 384),
    (64, 1, 100, 256, 128, 128), (100, 2, 2, 384, 96, 200), (128, 8, 32, 256, 128, 256),
    (1024, 1, 7, 128, 64, 40), (5, 2, 1024, 64, 32, 64),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,k,E,K,I,N", SHAPES)
def test_matches_definition(w4, T, k, E, K, I, N, dtype):
    ops = ref.make_experts(T + K, T, k, E, K, I, N, dtype)
    out = w4.w4a16_fp8_moe_mlp(*dev(ops))
    check(out, *ref.experts(*ops, dtype))
    assert w4.w4a16_device_status() == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_choices_that_are_none_or_repeated(w4, dtype):
    T, k, E, K, I, N = 24, 4, 6, 256, 128, 200
    ops = list(ref.make_experts(3, T, k, E, K, I, N, dtype))
    ids = ops[1]
    ids[0] = -1                    # a padded row
    ids[1, 1:] = -1
    ids[2] = 5                     # the same expert, four times
    ids[3:20, 0] = 5               # more of one than a tile holds
    ids[20, 2] = -1
    # what no row chooses does not matter
    ids[ids == 3] = 2
    ops[3].view(torch.uint8)[3] = 0x7f
    ops[4][3], ops[6][3] = float("nan"), float("inf")
    ops[2][0], ops[2][20, 2] = float("nan"), float("inf")
    out = w4.w4a16_fp8_moe_mlp(*dev(ops))
    assert bool((out[0] == 0).all())
    ops[2][0], ops[2][20, 2] = 0.0, 0.0
    check(out, *ref.experts(*ops, dtype))
    assert w4.w4a16_device_status() == 0
    ids[4, 1] = E                  # an id that is neither an expert nor -1 is reported
    ids[5, 0] = -2
    out = w4.w4a16_fp8_moe_mlp(*dev(ops))
    assert w4.w4a16_device_status() == 1024
    check(out, *ref.experts(*ops, dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_that_are_not_finite_keep_to_themselves(w4, dtype):
    T, k, E, K, I, N = 12, 2, 3, 256, 128, 96
    ops = list(ref.make_experts(8, T, k, E, K, I, N, dtype))
    ops[0][4, 7], ops[0][5, 200] = float("inf"), float("nan")
    out = ref.f64(w4.w4a16_fp8_moe_mlp(*dev(ops)))
    assert not np.isfinite(out[5]).any() and not np.isfinite(out[4]).all()
    clean = list(ops)
    clean[0] = ops[0].clone()
    clean[0][4:6] = 0.0
    want, bound = ref.experts(*clean, dtype)
    rows = [t for t in range(T) if t not in (4, 5)]
    assert np.all(np.abs(out - want)[rows] <= bound[rows])
    # a NaN weight: every row of the expert, and none of the others
    ops = list(ref.make_experts(9, T, k, E, K, I, N, dtype))
    ops[3].view(torch.uint8)[1, 3, 17] = 0xff
    out = ref.f64(w4.w4a16_fp8_moe_mlp(*dev(ops)))
    hit = (ops[1] == 1).any(1).numpy()
    assert hit.any() and np.isnan(out[hit]).all() and np.isfinite(out[~hit]).all()


def test_large_activations_and_gates(w4):
    # bf16 beyond fp16's range, and gates far on both sides of zero
    T, k, E, K, I, N = 6, 2, 4, 384, 160, 96
    ops = list(ref.make_experts(4, T, k, E, K, I, N, BF16))
    ops[0][0] *= 2.0 ** 30
    ops[0][1] *= 2.0 ** -40
    ops[0][2] *= 40
    out = w4.w4a16_fp8_moe_mlp(*dev(ops))
    check(out, *ref.experts(*ops, BF16))


def test_same_bits_every_time_on_any_stream_and_in_graphs(w4):
    a = dev(ref.make_experts(1, 16, 4, 12, 1024, 256, 512, BF16))
    b = dev(ref.make_experts(2, 40, 4, 12, 1024, 256, 512, BF16))
    want = [w4.w4a16_fp8_moe_mlp(*ops) for ops in (a, b)]
    for _ in range(10):
        for ops, w in zip((a, b), want):
            assert torch.equal(w4.w4a16_fp8_moe_mlp(*ops), w)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):  # two at a time
        got += [w4.w4a16_fp8_moe_mlp(*ops, stream=s) for ops, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    graphs, outs = [], []
    for ops in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(w4.w4a16_fp8_moe_mlp(*ops))
        graphs.append(graph)
    for s, graph in zip(streams, graphs):  # two replays at once
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    # other inputs under the same graph
    c = dev(ref.make_experts(7, 16, 4, 12, 1024, 256, 512, BF16))
    for to, new in zip(a, c):
        to.copy_(new)
    graphs[0].replay()
    assert torch.equal(outs[0], w4.w4a16_fp8_moe_mlp(*c))


def test_out_given_keeps_to_its_rows(w4):
    ops = dev(ref.make_experts(1, 5, 2, 4, 128, 64, 77, F16))
    want = w4.w4a16_fp8_moe_mlp(*ops)
    room = torch.full((7, 77), 3.0, dtype=F16, device=DEV)
    got = w4.w4a16_fp8_moe_mlp(*ops, out=room[1:6])
    assert torch.equal(got, want) and got.data_ptr() == room[1:6].data_ptr()
    assert bool((room[0] == 3).all()) and bool((room[6] == 3).all())
    empty = w4.w4a16_fp8_moe_mlp(ops[0][:0], ops[1][:0], ops[2][:0], *ops[3:])
    assert empty.shape == (0, 77)


def test_routed_layer_beside_the_4_bit_experts_calls(w4):
    """Router logits from a dense linear, the choice, the experts: as a decoder layer calls
    them, each step checked on what the one before left."""
    T, E, K, I, N, k = 19, 24, 256, 128, 256, 4
    ops = ref.make_experts(6, T, k, E, K, I, N, BF16)
    x, _, _, w1, s1, w2, s2 = dev(ops)
    router = torch.randn((E, K), generator=torch.Generator().manual_seed(1)).to(BF16)
    logits = w4.w4a16_dense_linear(x, router.to(DEV))
    ids, weights = w4.w4a16_moe_route(logits, k)
    want, p, _ = ref.route(logits, k, False, True)
    assert np.array_equal(ids.cpu().numpy(), want)
    out = w4.w4a16_fp8_moe_mlp(x, ids, weights, w1, s1, w2, s2)
    check(out, *ref.experts(ops[0], ids, weights, *ops[3:], BF16))
    # the same choice serves the 4-bit experts' calls
    srt, pos, off = w4.w4a16_moe_align(ids, E)
    assert int(off[-1]) == T * k
    assert w4.w4a16_device_status() == 0


def test_weights_beyond_32_bits(w4):
    # 8.6 GB of gate and up: the last expert's offset does not fit 32 bits
    T, E, K, I, N = 3, 1024, 4096, 1024, 40
    used = [0, 700, E - 1]
    x, ids, weights, w1, s1, w2, s2 = ref.make_experts(11, T, 1, 3, K, I, N, BF16)

    def spread(t):
        out = torch.zeros((E, *t.shape[1:]), dtype=t.dtype, device=DEV)
        for i, e in enumerate(used):
            out.view(torch.uint8 if t.element_size() == 1 else t.dtype)[e] = (
                t[i].view(torch.uint8) if t.element_size() == 1 else t[i]).to(DEV)
        return out

    ids[:, 0] = torch.tensor([0, 1, 2], dtype=torch.int32)
    far = torch.tensor(used, dtype=torch.int32)[ids.long()]
    out = w4.w4a16_fp8_moe_mlp(x.to(DEV), far.to(DEV), weights.to(DEV), *map(spread, (w1, s1, w2, s2)))
    check(out, *ref.experts(x, ids, weights, w1, s1, w2, s2, BF16))


@pytest.mark.parametrize("T", [1, 8])
def test_one_expert_for_everything(w4, T):
    # all choices on one expert: more slots than a tile of that many tokens holds
    k, E, K, I, N = 8, 16, 256, 128, 64
    ops = list(ref.make_experts(12, T, k, E, K, I, N, F16))
    ops[1][:] = 9
    check(w4.w4a16_fp8_moe_mlp(*dev(ops)), *ref.experts(*ops, F16))


@pytest.mark.parametrize("T,k", [(3, 2), (64, 8)])
def test_no_choice_at_all(w4, T, k):
    ops = list(ref.make_experts(13, T, k, 8, 128, 64, 48, BF16))
    ops[1][:] = -1
    out = w4.w4a16_fp8_moe_mlp(*dev(ops), out=torch.full((T, 48), 7.0, dtype=BF16, device=DEV))
    assert bool((out == 0).all())
