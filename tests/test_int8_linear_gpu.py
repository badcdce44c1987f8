"""LLM.int8 linear layer on the GPU: quantization of tokens, the product and its
gradient against 64-bit references (int8_cases.py)."""
import numpy as np
import pytest
import torch

import block_wise_bit_amd as dq4
from gpu_util import say
from int8_cases import (TYPES, backward64, check, linear64, quant64, to64, tokens, weight,
                        weight64)

pytestmark = pytest.mark.gpu

DTS = ("f16", "bf16")


def quant_checked(x, threshold, **given):
    codes, scales, outliers = dq4.dq4_int8_quant(x.cuda() if not x.is_cuda else x, threshold=threshold, **given)
    torch.cuda.synchronize()
    want, want_scales, listed = quant64(x, threshold)
    assert np.array_equal(codes.cpu().numpy().astype(np.int64), want)
    assert np.array_equal(to64(scales), want_scales, equal_nan=True)
    if listed is None:
        assert outliers is None
    else:
        assert np.array_equal(outliers.cpu().numpy().astype(np.int64), listed)
    return codes, scales, outliers


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("threshold", [0.0, 6.0])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 7), (1, 64), (1, 4096), (1, 8200), (1, 40001), (2, 1), (2, 8), (3, 9),
                                 (5, 63), (17, 64), (33, 1000), (64, 1377), (130, 4096), (7, 8192), (3, 20008),
                                 (700, 129), (2500, 72)])
def test_quant(dt, threshold, m, k):
    rng = np.random.default_rng(m * 1000 + k)
    quant_checked(tokens(rng, m, k, dt, outliers=min(5, k // 2)), threshold)


@pytest.mark.parametrize("m", [1, 2, 40])
def test_quant_at_the_largest_width(m):
    rng = np.random.default_rng(m)
    quant_checked(tokens(rng, m, 131071, "f16", outliers=3), 6.0)
    with pytest.raises(ValueError):
        dq4.dq4_int8_quant(torch.zeros((m, 131072), dtype=torch.float16, device="cuda"))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("m", [1, 3])
def test_quant_ties_and_borders(dt, m):
    """Quotients that lie on a half: x = (n + 1/2) s / 127 with s a multiple of
    127 (or three times one), and their neighbours in T."""
    eps = 2.0 ** -(10 if dt == "f16" else 7)
    halves = np.arange(-126, 127) + 0.5
    for s in (127.0, 254.0, 381.0, 508.0, 127.0 / 1024):
        v = halves * (s / 127.0)
        row = np.concatenate([[s, -s, 0.0, -0.0], v, v * (1 + eps), v * (1 - eps)])
        x = torch.from_numpy(np.tile(row, (m, 1))).to(TYPES[dt][0])
        quant_checked(x, 0.0)


@pytest.mark.parametrize("dt", DTS)
def test_quant_every_value_of_the_type(dt):
    """Every finite pattern of T under scales from the smallest to the largest."""
    t = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).view(TYPES[dt][0])
    t = t[torch.isfinite(t)]
    rows = []
    mags = torch.unique(t.abs().double())
    for s in (mags[1], mags[2], mags[100], mags[len(mags) // 3], mags[len(mags) // 2], mags[-2], mags[-1]):
        row = torch.where(t.double().abs() <= s, t.double(), torch.zeros(()).double())
        row[0] = s
        rows.append(row)
    quant_checked(torch.stack(rows).to(TYPES[dt][0]), 0.0)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("threshold", [0.0, 6.0, float("inf"), 1e-30, 3e38])
@pytest.mark.parametrize("m", [1, 4])
def test_quant_non_finite_and_empty_rows(dt, threshold, m):
    x = tokens(np.random.default_rng(3), m, 70, dt)
    x[0, 5], x[0, 6] = float("inf"), float("nan")
    if m > 1:
        x[1] = 0
        x[2, 64] = -torch.finfo(TYPES[dt][0]).max
        x[3, :] = float("-inf")
    quant_checked(x, threshold)


def test_quant_all_columns_outliers_and_none():
    rng = np.random.default_rng(8)
    for m, k in ((1, 300), (9, 300), (3, 9000), (2, 5000)):
        quant_checked(tokens(rng, m, k, "f16", outliers=k), 6.0)
        quant_checked(tokens(rng, m, k, "f16"), 6.0)


def test_quant_strided_rows_and_given_outputs():
    rng = np.random.default_rng(9)
    for m, k, pad in ((4, 40, 24), (5, 33, 7), (3, 64, 3)):
        wide = torch.full((m, k + pad), 77.0, dtype=torch.bfloat16)
        wide[:, :k] = tokens(rng, m, k, "bf16", outliers=2)
        dev = wide.cuda()
        buf = torch.full((m, k + pad + 1), 99, dtype=torch.int8, device="cuda")
        scales = torch.empty(m, device="cuda")
        quant_checked(dev[:, :k], 6.0, codes=buf[:, :k], scales=scales)
        assert bool((buf[:, k:] == 99).all())
    codes, scales, outliers = dq4.dq4_int8_quant(torch.zeros((0, 12), dtype=torch.float16, device="cuda"), 6.0)
    assert outliers.cpu().tolist() == [0] + [-1] * 12 and codes.shape == (0, 12)
    codes, scales, outliers = dq4.dq4_int8_quant(torch.zeros((3, 0), dtype=torch.float16, device="cuda"), 6.0)
    assert outliers.cpu().tolist() == [0] and scales.cpu().tolist() == [0.0] * 3


def linear_inputs(dt, m, n, k, outliers=0, bias=False, residual=False, seed=0):
    rng = np.random.default_rng(seed + m * 7 + n * 11 + k)
    x = tokens(rng, m, k, dt, outliers)
    codes, scales, listed = quant64(x, 6.0)
    CB, SCB = weight(rng, n, k)
    t = TYPES[dt][0]
    return dict(x=x, codes=codes, scales=scales, listed=listed, CB=CB, SCB=SCB,
                bias=torch.from_numpy(rng.standard_normal(n)).to(t) if bias else None,
                residual=torch.from_numpy(rng.standard_normal((m, n))).to(t) if residual else None)


def linear_checked(dt, c, mixed, what, **given):
    dev = {k: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v) for k, v in c.items()}
    codes = given.pop("codes", None)
    if codes is None:
        codes = dev["codes"].to(torch.int8).cuda()
    scales = dev["scales"].float().cuda()
    extra = {}
    cols = ()
    if mixed:
        extra = dict(x=c["x"].cuda(), outliers=torch.from_numpy(c["listed"]).int().cuda())
        cols = c["listed"][1:1 + c["listed"][0]]
    y = dq4.dq4_int8_linear(codes, scales, given.pop("CB", None) if "CB" in given else c["CB"].cuda(), c["SCB"].cuda(),
                            bias=None if c["bias"] is None else c["bias"].cuda(),
                            residual=None if c["residual"] is None else c["residual"].cuda(), dtype=TYPES[dt][0],
                            **extra, **given)
    want, bound = linear64(dt, c["codes"], c["scales"], c["CB"], c["SCB"],
                           None if c["bias"] is None else to64(c["bias"]),
                           None if c["residual"] is None else to64(c["residual"]), c["x"], cols)
    check(y, want, bound, what)
    return y


SHAPES = [(1, 1, 1), (1, 16, 64), (1, 33, 100), (1, 4096, 512), (2, 50, 16), (3, 17, 1000), (5, 300, 48), (16, 64, 128),
          (16, 9000, 80), (17, 130, 260), (31, 47, 1377), (33, 256, 192), (48, 100, 64), (64, 129, 1024),
          (64, 8200, 96), (65, 128, 64), (66, 1, 33), (100, 300, 1000), (128, 128, 128), (150, 1001, 1377),
          (200, 513, 48), (257, 260, 2376), (300, 1000, 640), (513, 700, 4096), (1030, 258, 80)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(dt, m, n, k):
    linear_checked(dt, linear_inputs(dt, m, n, k), False, f"{dt} {m}x{n}x{k}")
    linear_checked(dt, linear_inputs(dt, m, n, k, outliers=min(3, k), bias=True, residual=True), True,
                   f"{dt} {m}x{n}x{k} mixed")


@pytest.mark.parametrize("outliers", [1, 31, 32, 33, 64, 127, 128, 129, 200, 400])
@pytest.mark.parametrize("m", [1, 20, 64, 90, 300])
def test_linear_numbers_of_outliers(outliers, m):
    linear_checked("f16", linear_inputs("f16", m, 150, 400, outliers=outliers, bias=True), True, f"{m} {outliers}")


@pytest.mark.parametrize("m,n,k", [(2048, 4096, 4096), (1024, 1000, 14336), (300, 4096, 28672)])
def test_linear_large(m, n, k):
    linear_checked("bf16", linear_inputs("bf16", m, n, k, outliers=6, residual=True), True, f"{m}x{n}x{k}")


def test_linear_sums_at_the_32_bit_border():
    """All codes -128 or 127 over the largest width: the sum reaches 2^31 - 2^14."""
    k = 131071
    for m in (1, 70):
        c = dict(x=None, codes=np.full((m, k), -128), scales=np.full(m, 127.0), listed=None, bias=None, residual=None,
                 CB=torch.full((3, k), -128, dtype=torch.int8), SCB=torch.full((3,), 0.25))
        c["CB"][1] = 127
        linear_checked("bf16", c, False, f"largest sums, {m} rows")


def test_linear_strides_alignment_and_workspaces():
    for m, n, k, pad, skew in ((4, 40, 48, 16, 0), (7, 100, 64, 5, 1), (70, 130, 64, 16, 0), (70, 130, 64, 9, 3),
                               (90, 64, 100, 4, 2), (1, 70, 128, 0, 1), (33, 64, 65, 1, 0)):
        c = linear_inputs("f16", m, n, k, outliers=2, bias=True, residual=True)
        buf = torch.zeros(m * (k + pad) + skew, dtype=torch.int8, device="cuda")
        codes = buf[skew:].as_strided((m, k), (k + pad, 1))
        codes.copy_(torch.from_numpy(c["codes"]).to(torch.int8))
        wbuf = torch.zeros(n * k + 3, dtype=torch.int8, device="cuda")
        CB = wbuf[skew:skew + n * k].view(n, k)
        CB.copy_(c["CB"])
        out = torch.full((m, n + 6), 5.0, dtype=torch.float16, device="cuda")
        nbytes = dq4.dq4_int8_linear_workspace_bytes(n, k, m, True, codes=codes, CB=CB)
        ws = torch.randint(0, 256, (max(nbytes, 1),), dtype=torch.uint8, device="cuda")
        a = linear_checked("f16", dict(c), True, "strided", codes=codes, CB=CB, y=out[:, :n], workspace=ws)
        assert bool((out[:, n:] == 5).all())
        b = linear_checked("f16", dict(c), True, "dense")
        assert torch.equal(a, b)


def test_linear_in_place_residual_empty_sizes():
    c = linear_inputs("bf16", 9, 33, 64, residual=True)
    y = c["residual"].cuda()
    got = dq4.dq4_int8_linear(torch.from_numpy(c["codes"]).to(torch.int8).cuda(),
                              torch.from_numpy(c["scales"]).float().cuda(), c["CB"].cuda(), c["SCB"].cuda(),
                              residual=y, y=y)
    want, bound = linear64("bf16", c["codes"], c["scales"], c["CB"], c["SCB"], residual=to64(c["residual"]))
    check(got, want, bound, "in place")
    for m, n, k in ((0, 5, 6), (5, 0, 6), (5, 6, 0), (70, 6, 0)):
        i8 = torch.zeros((m, k), dtype=torch.int8, device="cuda")
        bias = torch.ones(n, dtype=torch.float16, device="cuda")
        y = dq4.dq4_int8_linear(i8, torch.zeros(m, device="cuda"), torch.zeros((n, k), dtype=torch.int8, device="cuda"),
                                torch.ones(n, device="cuda"), bias=bias)
        assert y.shape == (m, n) and bool((y == 1).all())


@pytest.mark.parametrize("m", [1, 5, 80])
def test_linear_rows_do_not_mix_non_finite(m):
    """A row with scale NaN, NaN and infinities in outlier columns: that row alone."""
    k, n = 96, 40
    x = tokens(np.random.default_rng(m), m, k, "f16", outliers=2)
    clean = x.clone()
    r = m // 2
    x[r, 7] = float("nan")
    codes, scales, outliers = dq4.dq4_int8_quant(x.cuda(), 6.0)
    CB, SCB = weight(np.random.default_rng(1), n, k)
    y = dq4.dq4_int8_linear(codes, scales, CB.cuda(), SCB.cuda(), x=x.cuda(), outliers=outliers).cpu()
    assert bool(torch.isnan(y[r]).all())
    keep = [i for i in range(m) if i != r]
    assert bool(torch.isfinite(y[keep]).all())
    codes, scales, _ = dq4.dq4_int8_quant(x.cuda())
    y = dq4.dq4_int8_linear(codes, scales, CB.cuda(), SCB.cuda()).cpu()
    assert bool(torch.isnan(y[r]).all()) and bool(torch.isfinite(y[keep]).all())
    codes, scales, _ = dq4.dq4_int8_quant(clean.cuda())
    z = dq4.dq4_int8_linear(codes, scales, CB.cuda(), SCB.cuda()).cpu()
    assert torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("m", [3, 100])
def test_linear_bad_outlier_lists(m):
    """Counts beyond the list and indices beyond the columns read nothing."""
    c = linear_inputs("f16", m, 40, 50)
    args = (torch.from_numpy(c["codes"]).to(torch.int8).cuda(), torch.from_numpy(c["scales"]).float().cuda(),
            c["CB"].cuda(), c["SCB"].cuda())
    for first, index, nan in ((1, 50, True), (1, -1, True), (1, 2 ** 30, True), (-5, 3, False), (51, 3, True),
                              (2 ** 31 - 1, 3, True)):
        listed = torch.full((51,), -1, dtype=torch.int32)
        listed[0], listed[1] = first, index
        y = dq4.dq4_int8_linear(*args, x=c["x"].cuda(), outliers=listed.cuda()).cpu()
        assert bool(torch.isnan(y).all()) == nan and bool(torch.isfinite(y).all()) != nan


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 64), (2, 33, 100), (17, 130, 1000), (64, 200, 128), (100, 77, 65),
                                   (150, 1001, 1377), (300, 512, 264), (37, 1000, 2376), (513, 640, 1024), (5, 40, 9)])
def test_backward(dt, m, n, k):
    rng = np.random.default_rng(m + n + k)
    CB, SCB = weight(rng, n, k)
    dy = torch.from_numpy(rng.standard_normal((m, n))).to(TYPES[dt][0])
    dx, dbias = dq4.dq4_int8_linear_backward(dy.cuda(), CB.cuda(), SCB.cuda(), bias_grad=True)
    (want, bound), (wb, bb) = backward64(dt, dy, CB, SCB)
    check(dx, want, bound, "dx")
    check(dbias, wb, bb, "dbias")
    only, none = dq4.dq4_int8_linear_backward(dy.cuda(), CB.cuda(), SCB.cuda())
    assert none is None and torch.equal(only, dx)


def test_backward_strides_misaligned_and_empty():
    rng = np.random.default_rng(4)
    for m, n, k, pad, skew in ((9, 40, 72, 3, 1), (140, 64, 128, 8, 0), (70, 33, 65, 5, 3), (20, 16, 24, 2, 4)):
        CB, SCB = weight(rng, n, k)
        wbuf = torch.zeros(n * k + 8, dtype=torch.int8, device="cuda")
        w = wbuf[skew:skew + n * k].view(n, k)
        w.copy_(CB)
        wide = torch.full((m, n + pad), 3.0, dtype=torch.float16, device="cuda")
        dy = torch.from_numpy(rng.standard_normal((m, n))).half()
        wide[:, :n] = dy.cuda()
        out = torch.full((m, k + pad), 9.0, dtype=torch.float16, device="cuda")
        ws = torch.randint(0, 256, (dq4.dq4_int8_linear_backward_workspace_bytes(n, k, m, wide[:, :n]),),
                           dtype=torch.uint8, device="cuda")
        dx, _ = dq4.dq4_int8_linear_backward(wide[:, :n], w, SCB.cuda(), dx=out[:, :k], workspace=ws)
        (want, bound), _ = backward64("f16", dy, CB, SCB)
        check(dx, want, bound, "dx")
        assert bool((out[:, k:] == 9).all())
    for m, n, k in ((0, 4, 5), (3, 0, 5), (3, 4, 0)):
        dx, db = dq4.dq4_int8_linear_backward(torch.ones((m, n), dtype=torch.float16, device="cuda"),
                                              torch.ones((n, k), dtype=torch.int8, device="cuda"),
                                              torch.ones(n, device="cuda"), bias_grad=True)
        assert dx.shape == (m, k) and bool((dx == 0).all()) and bool((db == m).all())


def test_backward_against_differences():
    """<dx, v> is the change of <dy, y> along v, for the 16-bit layer that the
    gradient is of: linear, so differences are exact up to rounding."""
    rng = np.random.default_rng(5)
    CB, SCB = weight(rng, 48, 80)
    w = weight64(CB, SCB, "f16")
    dy = torch.from_numpy(rng.standard_normal((6, 48))).half()
    dx, _ = dq4.dq4_int8_linear_backward(dy.cuda(), CB.cuda(), SCB.cuda())
    (_, bound), _ = backward64("f16", dy, CB, SCB)
    x = rng.standard_normal((6, 80))
    loss = lambda q: float((to64(dy) * (q @ w.T)).sum())  # noqa: E731
    for _ in range(4):
        v = rng.standard_normal((6, 80))
        h = 2.0 ** -10
        slope = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
        assert abs(slope - float((to64(dx) * v).sum())) <= float((bound * np.abs(v)).sum()) + 1e-8


def test_layer_as_used():
    """Quantize, multiply, go back: the calls in a row, on another stream, and as a
    graph that is replayed with new inputs."""
    rng = np.random.default_rng(6)
    m, n, k = 24, 200, 256
    CB, SCB = weight(rng, n, k)
    CBd, SCBd = CB.cuda(), SCB.cuda()
    x = tokens(rng, m, k, "f16", outliers=3).cuda()
    dy = torch.from_numpy(rng.standard_normal((m, n))).half().cuda()

    def layer(stream=None):
        codes, scales, outliers = dq4.dq4_int8_quant(x, 6.0, stream=stream)
        y = dq4.dq4_int8_linear(codes, scales, CBd, SCBd, residual=dy, x=x, outliers=outliers, stream=stream)
        dx, db = dq4.dq4_int8_linear_backward(dy, CBd, SCBd, bias_grad=True, stream=stream)
        return y, dx, db

    eager = layer()
    c64, s64, listed = quant64(x.cpu(), 6.0)
    want, bound = linear64("f16", c64, s64, CB, SCB, residual=to64(dy), x=x.cpu(), cols=listed[1:1 + listed[0]])
    check(eager[0], want, bound, "layer")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = layer(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for seed in range(4):
        new = tokens(np.random.default_rng(100 + seed), m, k, "f16", outliers=seed).cuda()
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        eager = layer()
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), seed
    say("four replays equal the eager calls")


def test_refusals():
    x = torch.zeros((4, 16), dtype=torch.float16, device="cuda")
    CB, SCB = torch.zeros((8, 16), dtype=torch.int8, device="cuda"), torch.zeros(8, device="cuda")
    codes, scales, outliers = dq4.dq4_int8_quant(x, 6.0)
    q, lin, back = dq4.dq4_int8_quant, dq4.dq4_int8_linear, dq4.dq4_int8_linear_backward
    y = torch.zeros((4, 8), dtype=torch.float16, device="cuda")
    for call in (lambda: q(x.float()), lambda: q(x, -1.0), lambda: q(x, float("nan")), lambda: q(x[0]),
                 lambda: q(x, 0.0, outliers=outliers), lambda: q(x, 6.0, outliers=outliers[:-1]),
                 lambda: q(x, 6.0, codes=codes.float()), lambda: q(x, 6.0, scales=scales[:2]),
                 lambda: q(x, 6.0, codes=x.view(torch.int8)[:, :16]), lambda: q(x.t()),
                 lambda: q(x, 6.0, workspace=torch.zeros(10, dtype=torch.uint8, device="cuda")),
                 lambda: lin(codes, scales, CB, SCB, x=x), lambda: lin(codes, scales, CB, SCB, outliers=outliers),
                 lambda: lin(codes[:, :8], scales, CB, SCB), lambda: lin(codes, scales[:3], CB, SCB),
                 lambda: lin(codes, scales, CB.float(), SCB), lambda: lin(codes, scales, CB, SCB.half()),
                 lambda: lin(codes, scales, CB, SCB, bias=y[0].float()), lambda: lin(codes, scales, CB, SCB, residual=y[:, :4]),
                 lambda: lin(codes, scales, CB, SCB, dtype=torch.float32), lambda: lin(codes, scales, CB.t(), SCB),
                 lambda: lin(codes, scales, CB, SCB, x=x.bfloat16(), outliers=outliers, dtype=torch.float16),
                 lambda: lin(codes, scales, CB, SCB, residual=y, y=torch.as_strided(y, (4, 8), (8, 1), 0)[:, :].view(torch.bfloat16)),
                 lambda: back(y.float(), CB, SCB), lambda: back(y[:, :4], CB, SCB), lambda: back(y, CB, SCB[:4]),
                 lambda: back(y, CB, SCB, dx=x[:3]), lambda: back(y, CB, SCB, dbias=SCB.half()),
                 lambda: back(y, CB, SCB, dbias=SCB), lambda: q(x.cpu()), lambda: lin(codes, scales, CB.cpu(), SCB),
                 lambda: lin(codes.cpu(), scales, CB, SCB)):
        with pytest.raises(ValueError):
            call()
