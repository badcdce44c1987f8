"""The LLM.int8 and mixture-of-experts calls where sizes, offsets and callers are out
of the ordinary: many rows of a weight to a workgroup, more than 2^32 elements, two
threads, several captured graphs, streams, shared memory."""
from __future__ import annotations

import threading

import numpy as np
import pytest

import block_wise_bit_amd as dq4

torch = pytest.importorskip("torch")

from block_wise_bit_amd import inputs  # noqa: E402
from int8_cases import TYPES, backward64, check, linear64, quant64, to64, tokens, weight  # noqa: E402
from moe_cases import Layer, moe64  # noqa: E402
from test_moe_gpu import choose, moe_checked, normal  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()
    yield
    torch.cuda.empty_cache()


def int8_columns_checked(m, n, k, dt="f16", outliers=0, seed=0):
    """The product over the whole weight, compared at the first, the last and some
    other output columns."""
    rng = np.random.default_rng(seed + m + n + k)
    x = tokens(rng, m, k, dt, outliers)
    codes, scales, listed = quant64(x, 6.0)
    torch.manual_seed(seed + n)
    CB = torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda")
    SCB = torch.rand(n, device="cuda") * 0.08 + 0.02
    extra, cols = {}, ()
    if outliers:
        extra = dict(x=x.cuda(), outliers=torch.from_numpy(listed).int().cuda())
        cols = listed[1:1 + listed[0]]
    y = dq4.dq4_int8_linear(torch.from_numpy(codes).to(torch.int8).cuda(), torch.from_numpy(scales).float().cuda(), CB,
                            SCB, dtype=TYPES[dt][0], **extra)
    pick = torch.from_numpy(np.unique(np.concatenate([np.arange(20), np.arange(n - 20, n),
                                                      rng.integers(0, n, 100)]))).cuda()
    want, bound = linear64(dt, codes, scales, CB[pick], SCB[pick], x=x, cols=cols)
    check(y[:, pick], want, bound, f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k,outliers", [
    (1, 8300, 8192, 3), (16, 8500, 1040, 0), (13, 4300, 4096, 2), (12, 8400, 14336, 0), (9, 8256, 20000, 5),
    (16, 8300, 8200, 3), (32, 8320, 4096, 40), (24, 9000, 8192, 0), (20, 8500, 12288, 2), (17, 8200, 1001, 0),
    (64, 9000, 2048, 7), (40, 8777, 4096, 0), (64, 8300, 4112, 3), (50, 8300, 5000, 2), (33, 16500, 512, 0),
    (3, 50000, 64, 0), (64, 50000, 128, 1), (1, 100, 131071, 4), (64, 33, 131056, 3)])
def test_int8_linear_many_rows_to_a_workgroup(m, n, k, outliers):
    int8_columns_checked(m, n, k, outliers=outliers)


@pytest.mark.parametrize("m,n,k", [(1024, 8200, 1040), (700, 16500, 512), (5000, 300, 200), (129, 40000, 64),
                                   (4100, 2100, 128)])
def test_int8_linear_many_tiles(m, n, k):
    int8_columns_checked(m, n, k, "bf16", outliers=2)


@pytest.mark.parametrize("m", [1, 20, 40, 70])
@pytest.mark.parametrize("k", [131056, 131071])
def test_int8_weight_of_more_than_2_to_32_bytes(m, k):
    int8_columns_checked(m, 40000, k, outliers=3)


@pytest.mark.parametrize("m,ld", [(3, (1 << 31) + 16), (40, (1 << 27) + 16), (100, 50000000), (100, 50000001)])
def test_int8_rows_that_lie_far_apart(m, ld):
    n, k = 70, 160
    rng = np.random.default_rng(m)
    x = tokens(rng, m, k, "bf16", 2)
    want_codes, want_scales, listed = quant64(x, 6.0)
    wide = torch.empty((m - 1) * ld + k, dtype=torch.bfloat16, device="cuda").as_strided((m, k), (ld, 1))
    wide.copy_(x)
    far = torch.empty((m - 1) * ld + k, dtype=torch.int8, device="cuda").as_strided((m, k), (ld, 1))
    codes, scales, outliers = dq4.dq4_int8_quant(wide, 6.0, codes=far)
    assert np.array_equal(codes.cpu().numpy().astype(np.int64), want_codes)
    assert np.array_equal(to64(scales), want_scales)
    CB, SCB = weight(rng, n, k)
    y = dq4.dq4_int8_linear(codes, scales, CB.cuda(), SCB.cuda(), x=wide, outliers=outliers)
    want, bound = linear64("bf16", want_codes, want_scales, CB, SCB, x=x, cols=listed[1:1 + listed[0]])
    check(y, want, bound, "far rows")


def test_int8_backward_of_a_far_weight():
    n, k = 40000, 131056
    for m in (2, 40):
        torch.manual_seed(m)
        CB = torch.zeros((n, k), dtype=torch.int8, device="cuda")
        SCB = torch.rand(n, device="cuda") * 0.08 + 0.02
        rows = torch.tensor([0, 5, 17000, 32779, 39999], device="cuda")  # the others are zeros
        CB[rows] = torch.randint(-128, 128, (5, k), dtype=torch.int8, device="cuda")
        dy = torch.randn((m, n), device="cuda").to(torch.bfloat16)
        dx, _ = dq4.dq4_int8_linear_backward(dy, CB, SCB)
        (want, bound), _ = backward64("bf16", dy[:, rows].cpu(), CB[rows].cpu(), SCB[rows].cpu())
        check(dx, want, bound, "far weight")


@pytest.mark.parametrize("m,n,k", [(3, 70000, 40), (1, 131072, 8), (128, 5000, 24), (129, 640, 264), (65, 33, 700),
                                   (33, 1000, 2376), (96, 24, 4099), (128, 4096, 1024), (16, 2048, 16384), (2, 17, 1)])
def test_int8_backward_few_tokens(m, n, k):
    rng = np.random.default_rng(m + n)
    CB, SCB = weight(rng, n, k)
    dy = normal(rng, (m, n), "f16")
    # what lies beside a row is not read, or has no part in the result
    for pad, skew in ((0, 0), (8, 0), (3, 1)):
        wide = torch.full((m, n + pad + skew), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, skew:skew + n] = dy.cuda()
        buf = torch.full((n * k + skew,), 77, dtype=torch.int8, device="cuda")
        CBd = buf[skew:].view(n, k)
        CBd.copy_(CB)
        dx, db = dq4.dq4_int8_linear_backward(wide[:, skew:skew + n], CBd, SCB.cuda(), bias_grad=True)
        (want, bound), (wb, bb) = backward64("f16", dy, CB, SCB)
        check(dx, want, bound, f"dx {m} {n} {k} {pad}")
        check(db, wb, bb, "dbias")


@pytest.mark.parametrize("m", [4, 40, 130])
def test_int8_backward_rows_do_not_mix(m):
    rng = np.random.default_rng(m)
    CB, SCB = weight(rng, 70, 90)
    dy = normal(rng, (m, 70), "bf16")
    clean, _ = dq4.dq4_int8_linear_backward(dy.cuda(), CB.cuda(), SCB.cuda())
    dy[2, 69] = float("nan")
    dy[3, 0] = float("inf")
    dx, _ = dq4.dq4_int8_linear_backward(dy.cuda(), CB.cuda(), SCB.cuda())
    keep = [i for i in range(m) if i not in (2, 3)]
    assert torch.equal(dx[keep], clean[keep]) and bool(torch.isnan(dx[2]).all())
    assert not bool(torch.isfinite(dx[3]).any())


# rows of multiples of 8 that are no multiples of 32, and larger layers
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("m,E,k,n_ff,n_in,bs", [
    (5, 3, 2, 24, 40, 32), (1, 3, 2, 40, 56, 32), (64, 4, 4, 72, 104, 64), (30, 4, 2, 24, 8, 32), (1, 2, 2, 8, 24, 32),
    (20, 3, 2, 1048, 1000, 32), (64, 3, 2, 1000, 2376, 64), (40, 5, 3, 520, 1032, 4096), (1, 4, 2, 1024, 2048, 64),
    (16, 2, 2, 2048, 4096, 64), (1, 2, 1, 4096, 2048, 128), (33, 2, 1, 4104, 520, 64)])
def test_moe_larger(dt, m, E, k, n_ff, n_in, bs):
    rng = np.random.default_rng(m + n_ff)
    layer = Layer(E, n_ff, n_in, bs, seed=20)
    ids, weights = choose(rng, m, E, k)
    moe_checked(dt, layer, normal(rng, (m, n_in), dt), ids, weights, residual=normal(rng, (m, n_in), dt),
                what=f"{dt} {m} {E} {k} {n_ff}x{n_in}")


@pytest.mark.parametrize("n_ff,n_in", [(64, 96), (24, 40), (33, 47)])
@pytest.mark.parametrize("m", [1, 5, 20, 64])
def test_moe_padded_rows_are_not_read(m, n_ff, n_in):
    """Rows without a valid expert hold NaN, as do the weights of ids that are none."""
    rng = np.random.default_rng(m)
    layer = Layer(5, n_ff, n_in, 32, seed=9)
    ids, weights = choose(rng, m, 5, 3)
    x, residual = normal(rng, (m, n_in), "f16"), normal(rng, (m, n_in), "f16")
    padded = np.arange(m) % 3 == (0 if m == 1 else 1)
    ids[padded] = -1
    ids[~padded, 1] = 5
    want, bound = moe64("f16", "silu", layer, x, ids, weights, residual)
    x[torch.from_numpy(padded)] = float("nan")
    weights[(ids < 0) | (ids > 4)] = np.nan
    y = dq4.dq4_moe_fused(*layer.device(), 5, n_ff, n_in, 32, x.cuda(), torch.from_numpy(ids).cuda(),
                          torch.from_numpy(weights).cuda(), residual=residual.cuda())
    check(y, want, bound, f"padded {m}")
    assert torch.equal(y.cpu()[torch.from_numpy(padded)], residual[torch.from_numpy(padded)])


def test_route_infinite_logits():
    """The softmax of an infinite logit is NaN, and masked experts stay out."""
    x, router = torch.ones((3, 8), dtype=torch.float16, device="cuda"), torch.ones((70, 8), dtype=torch.float16, device="cuda")
    bias = torch.zeros(70, device="cuda")
    bias[66], bias[2], bias[3] = float("inf"), float("-inf"), 1.0
    ids, weights = dq4.dq4_moe_route(x, router, 3, bias=bias)
    assert ids.cpu().tolist() == [[66, 3, 0]] * 3 and bool(torch.isnan(weights).all())
    bias[66] = -0.0  # as large as 0: the lower index first
    ids, weights = dq4.dq4_moe_route(x * 0, router, 4, bias=bias)
    assert ids.cpu().tolist() == [[3, 0, 1, 4]] * 3
    bias[:], bias[5], bias[66] = -1.0, -0.0, 0.0
    ids, weights = dq4.dq4_moe_route(x * 0, router, 2, bias=bias)
    assert ids.cpu().tolist() == [[5, 66]] * 3 and weights.cpu().tolist() == [[0.5, 0.5]] * 3


class Stacked:
    """The experts `of` of a stack that is drawn on the GPU, renumbered from 0."""

    def __init__(self, E, n_ff, n_in, bs, of):
        self.E, self.n_ff, self.n_in, self.blocksize, self.of = E, n_ff, n_in, bs, of
        self.sizes = (len(of), n_ff, n_in)
        n = E * n_ff * n_in
        assert n_ff * n_in % (bs * 256) == 0
        torch.manual_seed(3)
        self.dev, self.host = [], []
        for rows, cols in ((n_ff, n_in), (n_ff, n_in), (n_in, n_ff)):
            small = inputs.make_inputs(bs * 256, bs, "nf4", 0.03, seed=50 + len(self.dev))
            w = dq4.to_device(small)
            w["packed"] = torch.randint(0, 256, (n // 2,), dtype=torch.uint8, device="cuda")
            w["scale_codes"] = torch.randint(0, 256, (n // bs,), dtype=torch.uint8, device="cuda")
            w["nested_absmax"] = torch.rand(n // bs // 256, device="cuda") * 0.1
            self.dev.append(dict(w, offset=float(small.offset)))
            one = rows * cols
            cut = lambda t, size: torch.cat([t[e * size:(e + 1) * size] for e in of]).cpu().numpy()  # noqa: E731
            self.host.append(inputs.NestedInputs(
                cut(w["packed"], one // 2), cut(w["scale_codes"], one // bs), cut(w["nested_absmax"], one // bs // 256),
                small.scale_codebook, small.codebook4, small.offset, one * len(of), bs, n_rows=rows * len(of), n_cols=cols))

    matrices = Layer.matrices


@pytest.mark.parametrize("E,n_ff,n_in", [(512, 4096, 4608), (512, 4128, 4096)])
def test_moe_weights_of_more_than_2_to_32_bytes(E, n_ff, n_in):
    layer = Stacked(E, n_ff, n_in, 64, (0, 260, E - 1))
    assert E * n_ff * n_in // 2 > 1 << 32
    for m in (1, 16, 40):
        rng = np.random.default_rng(m)
        ids, weights = choose(rng, m, 3, 2)
        x = normal(rng, (m, n_in), "bf16")
        y = dq4.dq4_moe_fused(*layer.dev, E, n_ff, n_in, 64, x.cuda(),
                              torch.from_numpy(np.array(layer.of, np.int32)[ids]).cuda(), torch.from_numpy(weights).cuda())
        want, bound = moe64("bf16", "silu", layer, x, ids, weights)
        check(y, want, bound, f"far experts, {m}")


def layers(m, seed=0):
    """A layer of each kind with its inputs: {name: a call that takes stream= and
    workspace=, and the workspace's bytes}."""
    rng = np.random.default_rng(seed + m)
    n, k, E, n_ff, n_in = 300, 520, 6, 136, 200
    CB, SCB = (t.cuda() for t in weight(rng, n, k))
    x, dy = tokens(rng, m, k, "f16", 3).cuda(), normal(rng, (m, n), "f16").cuda()
    codes, scales, outliers = dq4.dq4_int8_quant(x, 6.0)
    layer = Layer(E, n_ff, n_in, 32, seed=30)
    dev = layer.device()
    z, router = normal(rng, (m, n_in), "bf16").cuda(), normal(rng, (E, n_in), "bf16").cuda()
    ids, weights = dq4.dq4_moe_route(z, router, 2)
    torch.cuda.synchronize()
    calls = {
        "quant": lambda **g: dq4.dq4_int8_quant(x, 6.0, **g),
        "linear": lambda **g: (dq4.dq4_int8_linear(codes, scales, CB, SCB, x=x, outliers=outliers, **g),),
        "backward": lambda **g: dq4.dq4_int8_linear_backward(dy, CB, SCB, bias_grad=True, **g),
        "route": lambda **g: dq4.dq4_moe_route(z, router, 2, **g),
        "experts": lambda **g: (dq4.dq4_moe_fused(*dev, E, n_ff, n_in, 32, z, ids, weights, residual=z, **g),),
    }
    return calls, (x, dy, z)


NAMES = ("quant", "linear", "backward", "route", "experts")


def equal(a, b):
    return all(p is q is None or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("m,name", [(m, name) for m in (1, 40, 150) for name in NAMES
                                    if m <= 64 or name not in ("route", "experts")])
def test_allocations_come_from_the_given_stream(m, name, monkeypatch):
    call = layers(m)[0][name]
    side = torch.cuda.Stream()
    want = call()
    torch.cuda.synchronize()
    made = []
    empty = torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        made.append((torch.cuda.current_stream().cuda_stream, t.numel()))
        return t
    monkeypatch.setattr(torch, "empty", spy)
    got = call(stream=side)
    monkeypatch.undo()
    side.synchronize()
    assert [s for s, size in made if size]
    assert all(s == side.cuda_stream for s, size in made if size)
    assert equal(got, want)


@pytest.mark.parametrize("m", [1, 40])
def test_two_threads_at_once(m):
    """Each with its own stream and its own inputs."""
    results, errors = {}, []
    sets = {seed: layers(m, seed)[0] for seed in (1, 2)}
    want = {seed: {name: calls[name]() for name in NAMES} for seed, calls in sets.items()}
    torch.cuda.synchronize()

    def run(seed):
        try:
            side = torch.cuda.Stream()
            for _ in range(20):
                results[seed] = {name: sets[seed][name](stream=side) for name in NAMES}
            side.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(seed,)) for seed in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for seed in sets:
        for name in NAMES:
            assert equal(results[seed][name], want[seed][name]), (seed, name)


@pytest.mark.parametrize("m", [1, 2, 20, 64])
def test_two_graphs_that_share_a_workspace(m):
    """A call's workspace holds nothing from one call to the next: two captured
    graphs and eager calls take turns with one."""
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    (a, fresh_a), (b, _) = layers(m, 5), layers(m, 6)
    graphs = []
    for calls in (a, b):
        for name in NAMES:
            calls[name](workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = {name: calls[name](workspace=ws) for name in NAMES}
        graphs.append((g, held, calls))
    rng = np.random.default_rng(9)
    for turn in range(3):
        for t in fresh_a:
            t.copy_(normal(rng, tuple(t.shape), "bf16" if t.dtype == torch.bfloat16 else "f16") * 3)
        for g, held, calls in graphs:
            g.replay()
            torch.cuda.synchronize()
            for name in NAMES:
                assert equal(held[name], calls[name]()), (turn, name)


def test_two_workspaces_at_once_on_two_streams():
    """The same call on two streams, each with memory of its own, in flight together."""
    calls, _ = layers(40, 7)
    want = {name: calls[name]() for name in NAMES}
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [[calls[name](stream=s) for s in sides for name in NAMES] for _ in range(10)]
    torch.cuda.synchronize()
    for row in got:
        for i, r in enumerate(row):
            assert equal(r, want[NAMES[i % len(NAMES)]])


def test_shared_memory_is_refused():
    """An output or a workspace that shares memory with what a call reads."""
    pool = torch.zeros(1 << 18, dtype=torch.uint8, device="cuda")
    half = lambda at, *shape: pool[at:at + 2 * int(np.prod(shape))].view(torch.float16).view(*shape)  # noqa: E731
    i8 = lambda at, *shape: pool[at:at + int(np.prod(shape))].view(torch.int8).view(*shape)  # noqa: E731
    f32 = lambda at, n: pool[at:at + 4 * n].view(torch.float32)  # noqa: E731
    i32 = lambda at, *shape: pool[at:at + 4 * int(np.prod(shape))].view(torch.int32).view(*shape)  # noqa: E731
    x, far = half(0, 4, 32), pool[32768:]
    CB, SCB = i8(1024, 16, 32), f32(2048, 16)
    codes, scales = i8(4096, 4, 32), f32(5120, 4)
    dy = half(6144, 4, 16)
    router = half(8192, 3, 32)
    ids, weights = i32(12288, 4, 2), pool[12800:12832].view(torch.float32).view(4, 2)
    layer = Layer(3, 16, 32, 32)
    dev = layer.device()

    dq4.dq4_int8_quant(x, 6.0, codes=i8(16384, 4, 32), workspace=far)
    dq4.dq4_int8_linear(codes, scales, CB, SCB, dtype=torch.float16, workspace=far)
    dq4.dq4_int8_linear_backward(dy, CB, SCB, workspace=far)
    dq4.dq4_moe_route(x, router, 2, ids=ids, weights=weights, workspace=far)
    dq4.dq4_moe_fused(*dev, 3, 16, 32, 32, x, ids, weights, workspace=far)
    torch.cuda.synchronize()
    for call in (lambda: dq4.dq4_int8_quant(x, 6.0, codes=i8(16, 4, 32)),
                 lambda: dq4.dq4_int8_quant(x, 6.0, scales=f32(64, 4)),
                 lambda: dq4.dq4_int8_quant(x, 6.0, workspace=pool),
                 lambda: dq4.dq4_int8_quant(x, 6.0, codes=codes, scales=f32(4096 + 64, 4)),
                 lambda: dq4.dq4_int8_quant(x, 6.0, codes=codes, workspace=pool[4096:8192]),
                 lambda: dq4.dq4_int8_linear(codes, scales, CB, SCB, y=half(1024, 4, 16)),
                 lambda: dq4.dq4_int8_linear(codes, scales, CB, SCB, y=half(4096, 4, 16)),
                 lambda: dq4.dq4_int8_linear(codes, scales, CB, SCB, y=half(16384, 4, 16), workspace=pool[2048:]),
                 lambda: dq4.dq4_int8_linear_backward(dy, CB, SCB, dx=half(6144, 4, 32)),
                 lambda: dq4.dq4_int8_linear_backward(dy, CB, SCB, dx=half(1024, 4, 32)),
                 lambda: dq4.dq4_int8_linear_backward(dy, CB, SCB, workspace=pool),
                 lambda: dq4.dq4_moe_route(x, router, 2, weights=pool[0:32].view(torch.float32).view(4, 2)),
                 lambda: dq4.dq4_moe_route(x, router, 2, ids=i32(8192, 4, 2)),
                 lambda: dq4.dq4_moe_route(x, router, 2, ids=ids, weights=ids.view(torch.float32)),
                 lambda: dq4.dq4_moe_route(x, router, 2, workspace=pool),
                 lambda: dq4.dq4_moe_fused(*dev, 3, 16, 32, 32, x, ids, weights, y=x),
                 lambda: dq4.dq4_moe_fused(*dev, 3, 16, 32, 32, x, ids, weights, y=half(12800, 4, 32)),
                 lambda: dq4.dq4_moe_fused(*dev, 3, 16, 32, 32, x, ids, weights, workspace=pool),
                 lambda: dq4.dq4_moe_fused(*dev, 3, 16, 32, 32, x, ids, weights, y=half(40000, 4, 32), workspace=far)):
        with pytest.raises(ValueError):
            call()
