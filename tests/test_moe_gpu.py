"""Mixture-of-experts layer on the GPU: the router and the experts' products
against 64-bit references (moe_cases.py)."""
import numpy as np
import pytest
import torch

import block_wise_bit_amd as dq4
from gpu_util import say
from moe_cases import TYPES, Layer, check, moe64, route64, to64

pytestmark = pytest.mark.gpu

DTS = ("f16", "bf16")


def coarse(rng, shape, dt):
    """Multiples of 2^-6 below 4: products and their sums are exact in FP64, and
    different experts' logits differ by 2^-12 or are equal."""
    return torch.from_numpy(rng.integers(-200, 201, shape) / 64.0).to(TYPES[dt][0])


def route_checked(x, router, top_k, bias=None, renormalize=True, **given):
    ids, weights = dq4.dq4_moe_route(x.cuda() if not x.is_cuda else x, router.cuda(), top_k,
                                     bias=None if bias is None else torch.from_numpy(bias).cuda(),
                                     renormalize=renormalize, **given)
    want, w, bound = route64(x, router, top_k, bias, renormalize)
    assert np.array_equal(ids.cpu().numpy(), want)
    got = to64(weights)
    nan = np.isnan(w)
    assert np.array_equal(np.isnan(got), nan)
    err = np.abs(np.where(nan, 0, got - w))
    assert (err <= np.where(nan, 0, bound)).all(), float((err / np.maximum(bound, 1e-300)).max())
    return ids, weights


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("m,E,k,n", [(1, 1, 1, 1), (1, 8, 2, 64), (3, 4, 4, 7), (1, 64, 8, 2048), (16, 64, 8, 512),
                                     (5, 65, 3, 1001), (64, 128, 8, 520), (2, 512, 16, 96), (300, 16, 4, 2376),
                                     (2500, 8, 2, 40), (7, 100, 16, 4099)])
def test_route(dt, m, E, k, n):
    rng = np.random.default_rng(m + E + n)
    x, router = coarse(rng, (m, n), dt), coarse(rng, (E, n), dt)
    for renormalize in (True, False):
        route_checked(x, router, k, renormalize=renormalize)
    route_checked(x, router, k, bias=rng.integers(-50, 51, E).astype(np.float32) / 16)


def test_route_ties_go_to_the_lower_index():
    x = torch.ones((3, 16), dtype=torch.float16)
    router = torch.zeros((40, 16), dtype=torch.float16)
    router[[7, 21, 22, 39]] = 1
    ids, weights = route_checked(x, router, 6)
    assert ids[0].cpu().tolist() == [7, 21, 22, 39, 0, 1]


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_masks_and_non_finite_logits(renormalize):
    rng = np.random.default_rng(2)
    x, router = coarse(rng, (6, 24), "bf16"), coarse(rng, (9, 24), "bf16")
    bias = np.zeros(9, np.float32)
    bias[[1, 3, 4, 5, 6, 8]] = -np.inf
    ids, weights = route_checked(x, router, 5, bias=bias, renormalize=renormalize)  # three experts are left
    assert bool((ids[:, 3:] == -1).all()) and bool((weights[:, 3:] == 0).all())
    ids, weights = route_checked(x, router, 2, bias=np.full(9, -np.inf, np.float32), renormalize=renormalize)
    assert bool((ids == -1).all()) and bool((weights == 0).all())
    bias = np.full(9, -3.4028235e38, np.float32)  # the type's lowest value masks too, but leaves an order
    bias[2] = 0
    route_checked(x, router, 2, bias=bias, renormalize=renormalize)
    bias = np.zeros(9, np.float32)
    bias[4] = np.nan
    ids, weights = route_checked(x, router, 9, bias=bias, renormalize=renormalize)
    assert bool((ids[:, 8] == 4).all()) and bool(torch.isnan(weights).all())
    x[2, 3] = float("nan")
    ids, weights = route_checked(x, router, 3, renormalize=renormalize)
    assert ids[2].cpu().tolist() == [0, 1, 2] and bool(torch.isfinite(weights[[0, 1, 3, 4, 5]]).all())


def test_route_strided_rows_given_outputs_and_no_columns():
    rng = np.random.default_rng(3)
    wide = coarse(rng, (5, 70), "f16").cuda()
    router = coarse(rng, (6, 65), "f16")
    ids, weights = torch.empty((5, 2), dtype=torch.int32, device="cuda"), torch.empty((5, 2), device="cuda")
    got = route_checked(wide[:, 3:68], router, 2, ids=ids, weights=weights)
    assert got[0] is ids and got[1] is weights
    ids, weights = dq4.dq4_moe_route(torch.zeros((2, 0), dtype=torch.float16, device="cuda"),
                                     torch.zeros((4, 0), dtype=torch.float16, device="cuda"), 2)
    assert ids.cpu().tolist() == [[0, 1]] * 2 and weights.cpu().tolist() == [[0.5, 0.5]] * 2
    ids, weights = dq4.dq4_moe_route(wide[:0, :65], router.cuda(), 2)
    assert ids.shape == (0, 2) and weights.shape == (0, 2)


def choose(rng, m, E, k):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(m)]).astype(np.int32) if m else np.zeros((0, k), np.int32)
    w = rng.random((m, k)).astype(np.float32)
    return ids, (w / np.maximum(w.sum(axis=1, keepdims=True), 1e-9)).astype(np.float32)


def moe_checked(dt, layer, x, ids, weights, act="silu", residual=None, what="", dev=None, **given):
    E, n_ff, n_in = layer.sizes
    gate, up, down = dev or layer.device()
    y = dq4.dq4_moe_fused(gate, up, down, E, n_ff, n_in, layer.blocksize, x if x.is_cuda else x.cuda(),
                          torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(), activation=act,
                          residual=None if residual is None else residual.cuda(), **given)
    want, bound = moe64(dt, act, layer, x, ids, weights, residual)
    check(y, want, bound, what)
    return y


def normal(rng, shape, dt):
    return torch.from_numpy(rng.standard_normal(shape)).to(TYPES[dt][0])


SHAPES = [  # m, experts, top_k, n_ff, n_in, blocksize
    (1, 1, 1, 16, 32, 32), (1, 4, 2, 64, 64, 64), (1, 8, 2, 32, 96, 32), (1, 8, 8, 512, 1024, 64),
    (3, 4, 2, 48, 160, 64), (5, 3, 3, 7, 9, 32), (2, 5, 2, 33, 65, 32), (16, 8, 2, 128, 512, 64),
    (16, 16, 4, 100, 236, 128), (17, 4, 2, 64, 128, 64), (33, 2, 2, 96, 64, 32), (40, 9, 3, 257, 130, 256),
    (64, 2, 1, 64, 96, 64), (64, 32, 8, 40, 72, 64), (64, 4, 4, 520, 1030, 1024), (20, 64, 16, 17, 31, 32),
    (64, 6, 2, 1000, 2376, 128), (1, 3, 1, 2050, 4104, 4096), (9, 4, 2, 1024, 1376, 32), (64, 3, 2, 544, 672, 32),
]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("m,E,k,n_ff,n_in,bs", SHAPES)
def test_experts(dt, m, E, k, n_ff, n_in, bs):
    rng = np.random.default_rng(m + E + n_ff)
    layer = Layer(E, n_ff, n_in, bs)
    ids, weights = choose(rng, m, E, k)
    act = ("silu", "gelu", "gelu_tanh", "relu")[(m + E + k) % 4]
    residual = normal(rng, (m, n_in), dt) if (m + k) % 2 else None
    moe_checked(dt, layer, normal(rng, (m, n_in), dt), ids, weights, act, residual, f"{dt} {m} {E} {k} {n_ff}x{n_in}")


@pytest.mark.parametrize("n_ff,n_in", [(64, 96), (33, 47)])
@pytest.mark.parametrize("m", [1, 6, 16, 40, 64])
def test_experts_odd_choices(m, n_ff, n_in):
    """Everybody on one expert, nobody on any, padded rows, ids out of range, an id
    twice in a row, weights of zero."""
    rng = np.random.default_rng(m)
    layer = Layer(7, n_ff, n_in, 32, seed=4)
    dev = layer.device()
    x, residual = normal(rng, (m, n_in), "f16"), normal(rng, (m, n_in), "f16")
    ids, weights = choose(rng, m, 7, 3)
    cases = [np.full((m, 3), 5), np.full((m, 3), -1), np.where(np.arange(m)[:, None] % 2, ids, -1),
             np.where(ids == 2, 7, np.where(ids == 3, 2 ** 31 - 1, ids)), np.stack([ids[:, 0], ids[:, 0], ids[:, 1]], 1),
             np.stack([ids[:, 0], np.full(m, -7), ids[:, 0]], 1)]
    for i, c in enumerate(cases):
        y = moe_checked("f16", layer, x, c.astype(np.int32), weights, residual=residual if i % 2 else None,
                        what=f"choice {i}", dev=dev)
        if i == 1:
            assert torch.equal(y.cpu(), residual)
    none = moe_checked("f16", layer, x, np.full((m, 3), -1, np.int32), weights, dev=dev)
    assert bool((none == 0).all())


def test_experts_rows_do_not_mix_non_finite():
    """NaN and infinities in one token, NaN in one expert that others did not choose
    and a NaN weight stay where they are."""
    rng = np.random.default_rng(5)
    layer = Layer(4, 48, 64, 32, seed=6)
    gate, up, down = layer.device()
    for m in (4, 30):
        x = normal(rng, (m, 64), "bf16")
        ids, weights = choose(rng, m, 3, 2)  # expert 3 belongs to token 2 alone
        ids[2] = 3
        args = (4, 48, 64, 32)
        clean = dq4.dq4_moe_fused(gate, up, down, *args, x.cuda(), torch.from_numpy(ids).cuda(),
                                  torch.from_numpy(weights).cuda()).cpu()
        x[1, 5] = float("nan")
        weights[0, 0] = np.nan
        bad = dict(gate, nested_absmax=gate["nested_absmax"].clone())
        # 64 x 48 x 4 elements in blocks of 32 fill two groups of 256 blocks; expert 3 lies in the second
        first = 3 * 48 * 64 // 32 // 256
        assert first == 1
        codes = bad["scale_codes"] = gate["scale_codes"].clone()
        book = bad["scale_codebook"] = gate["scale_codebook"].clone()
        codes[codes == 255] = 254
        codes[3 * 48 * 64 // 32:] = 255
        book[255] = float("nan")
        y = dq4.dq4_moe_fused(bad, up, down, *args, x.cuda(), torch.from_numpy(ids).cuda(),
                              torch.from_numpy(weights).cuda()).cpu()
        for t in (0, 1, 2):
            assert bool(torch.isnan(y[t]).all())
        assert bool(torch.isfinite(y[3:]).all())
        del clean


def test_experts_strides_alignment_workspace():
    rng = np.random.default_rng(7)
    for m, E, k, n_ff, n_in, skew in ((5, 4, 2, 64, 96, 1), (20, 5, 2, 64, 64, 2), (3, 3, 2, 50, 70, 3), (2, 2, 2, 32, 32, 4)):
        layer = Layer(E, n_ff, n_in, 64, seed=8)
        dev = layer.device()
        for w in dev:
            buf = torch.zeros(w["packed"].numel() + 8, dtype=torch.uint8, device="cuda")
            view = buf[skew:skew + w["packed"].numel()]
            view.copy_(w["packed"])
            w["packed"] = view
        wide = torch.full((m, n_in + 5), 3.0, dtype=torch.float16, device="cuda")
        x = normal(rng, (m, n_in), "f16")
        wide[:, 1:1 + n_in] = x.cuda()
        out = torch.full((m, n_in + 3), 9.0, dtype=torch.float16, device="cuda")
        ids, weights = choose(rng, m, E, k)
        size = dq4.dq4_moe_fused_workspace_bytes(E, n_ff, n_in, m, k)
        for fill in (0, 255):
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            a = moe_checked("f16", layer, wide[:, 1:1 + n_in], ids, weights, what="strided", dev=dev, y=out[:, :n_in],
                            workspace=ws)
            assert bool((out[:, n_in:] == 9).all())
        b = moe_checked("f16", layer, x, ids, weights, what="dense", dev=dev)
        assert torch.equal(a, b)


def test_experts_empty_sizes_and_residual_in_place():
    rng = np.random.default_rng(9)
    layer = Layer(3, 32, 64, 32, seed=10)
    x, r = normal(rng, (4, 64), "bf16"), normal(rng, (4, 64), "bf16")
    ids, weights = choose(rng, 4, 3, 2)
    y = r.cuda()
    gate, up, down = layer.device()
    got = dq4.dq4_moe_fused(gate, up, down, 3, 32, 64, 32, x.cuda(), torch.from_numpy(ids).cuda(),
                            torch.from_numpy(weights).cuda(), residual=y, y=y)
    want, bound = moe64("bf16", "silu", layer, x, ids, weights, r)
    check(got, want, bound, "in place")
    none = dq4.dq4_moe_fused(gate, up, down, 3, 0, 64, 32, x.cuda(), torch.from_numpy(ids).cuda(),
                             torch.from_numpy(weights).cuda(), residual=r.cuda())
    assert torch.equal(none.cpu(), r)
    none = dq4.dq4_moe_fused(gate, up, down, 3, 32, 64, 32, x.cuda()[:0], torch.from_numpy(ids[:0]).cuda(),
                             torch.from_numpy(weights[:0]).cuda())
    assert none.shape == (0, 64)


def test_decoder_block_as_used():
    """An LLM.int8 projection, the router and the experts of a decoder block, eager,
    on another stream, and as a graph that is replayed with new inputs."""
    rng = np.random.default_rng(11)
    m, E, k, n_ff, n_in = 6, 8, 2, 96, 128
    layer = Layer(E, n_ff, n_in, 64, seed=12)
    gate, up, down = layer.device()
    CB = torch.from_numpy(rng.integers(-127, 128, (n_in, n_in), dtype=np.int8)).cuda()
    SCB = torch.full((n_in,), 0.05, device="cuda")
    router = normal(rng, (E, n_in), "f16").cuda()
    a, x = normal(rng, (m, n_in), "f16").cuda(), normal(rng, (m, n_in), "f16").cuda()

    def block(stream=None):
        codes, scales, outliers = dq4.dq4_int8_quant(a, 3.0, stream=stream)
        z = dq4.dq4_int8_linear(codes, scales, CB, SCB, residual=x, x=a, outliers=outliers, stream=stream)
        ids, weights = dq4.dq4_moe_route(z, router, k, stream=stream)
        y = dq4.dq4_moe_fused(gate, up, down, E, n_ff, n_in, 64, z, ids, weights, residual=z, stream=stream)
        return z, ids, weights, y

    z, ids, weights, y = block()
    want, bound = moe64("f16", "silu", layer, z, ids.cpu().numpy(), weights.cpu().numpy(), z)
    check(y, want, bound, "block")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = block(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip((z, ids, weights, y), other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block()
    for seed in range(4):
        new = np.random.default_rng(50 + seed)
        a.copy_(normal(new, (m, n_in), "f16"))
        x.copy_(normal(new, (m, n_in), "f16"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(block(), held)), seed
    say("four replays equal the eager calls")


def test_refusals():
    layer = Layer(3, 32, 64, 32, seed=10)
    gate, up, down = layer.device()
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    ids, weights = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    router = torch.zeros((3, 64), dtype=torch.float16, device="cuda")

    def moe(g=gate, u=up, d=down, E=3, n_ff=32, n_in=64, bs=32, x=x, ids=ids, weights=weights, **k):
        return dq4.dq4_moe_fused(g, u, d, E, n_ff, n_in, bs, x, ids, weights, **k)

    moe()
    many = torch.zeros((65, 64), dtype=torch.float16, device="cuda")
    for call in (lambda: moe(E=4), lambda: moe(E=0), lambda: moe(bs=48), lambda: moe(x=x.float()), lambda: moe(x=x[:, :32]),
                 lambda: moe(ids=ids.long()), lambda: moe(ids=ids[:3]), lambda: moe(weights=weights.half()),
                 lambda: moe(weights=weights[:, :1]), lambda: moe(activation="none"), lambda: moe(residual=x[:2]),
                 lambda: moe(y=x), lambda: moe(residual=x, y=x.view(torch.bfloat16)), lambda: moe(x=x.cpu()),
                 lambda: moe(x=many, ids=ids.new_zeros((65, 2)), weights=weights.new_zeros((65, 2))),
                 lambda: moe(ids=ids.new_zeros((4, 17)), weights=weights.new_zeros((4, 17))),
                 lambda: moe(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                 lambda: moe(nested_blocksize=128), lambda: moe(ids=ids.t().contiguous().t()),
                 lambda: dq4.dq4_moe_route(x, router, 0), lambda: dq4.dq4_moe_route(x, router, 4),
                 lambda: dq4.dq4_moe_route(x.float(), router, 2), lambda: dq4.dq4_moe_route(x, router.bfloat16(), 2),
                 lambda: dq4.dq4_moe_route(x, router[:, :32], 2), lambda: dq4.dq4_moe_route(x, router, 2, bias=router[:, 0]),
                 lambda: dq4.dq4_moe_route(x, x.new_zeros((513, 64)), 2), lambda: dq4.dq4_moe_route(x, x.new_zeros((20, 64)), 17),
                 lambda: dq4.dq4_moe_route(x, router, 2, ids=ids.long()), lambda: dq4.dq4_moe_route(x.cpu(), router, 2)):
        with pytest.raises(ValueError):
            call()
