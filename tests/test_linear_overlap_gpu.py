"""Overlaps that the fused calls' binding refuses: a caller's workspace with any
matrix or any part of a weight, and an output with any part of a weight.  (The
overlaps of matrices among each other: test_linear_fused_gpu.py.)"""
from __future__ import annotations

import pytest

import block_wise_bit_amd as dq4
from block_wise_bit_amd import inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

N_OUT, N_IN, M = 64, 128, 4
BYTES = 1 << 20   # more workspace than any of these calls asks for


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()


PARTS = ["packed", "scale_codes", "nested_absmax", "scale_codebook", "codebook4"]


def pool_weight(seed):
    """A weight whose parts lie in one pool of bytes, 64 KiB apart, behind a
    free 1 MiB: (pool, weight)."""
    x = inputs.make_inputs(N_OUT * N_IN, 64, "nf4", 0.03, seed=seed, n_rows=N_OUT, n_cols=N_IN)
    pool = torch.zeros(BYTES + 6 * 65536, dtype=torch.uint8, device="cuda")
    w = {}
    for i, (name, t) in enumerate(dq4.to_device(x).items()):
        raw = t.view(torch.uint8).reshape(-1)
        at = BYTES + i * 65536
        pool[at:at + raw.numel()] = raw
        w[name] = pool[at:at + raw.numel()].view(t.dtype)
    return pool, dict(w, offset=float(x.offset))


def matrix(pool, at, rows, cols):
    return pool[at:at + 2 * rows * cols].view(torch.bfloat16).view(rows, cols)


def four_calls(w, up, t):
    """{name: (the call, its inputs, its outputs)} with every matrix from t(rows, cols)."""
    sizes = dict(n_out=N_OUT, n_in=N_IN, blocksize=64)
    x, dy, pre, g, u = t(M, N_IN), t(M, N_OUT), t(M, N_OUT), t(M, N_OUT), t(M, N_OUT)
    return {
        "linear": (lambda **k: dq4.dq4_linear_fused(**w, **sizes, **dict(dict(x=x, residual=dy, bias=pre[0],
                                                                              activation="silu"), **k)),
                   ["x", "residual"], ["y", "pre"]),
        "linear backward": (lambda **k: dq4.dq4_linear_fused_backward(
            **w, **sizes, **dict(dict(dy=dy, pre=pre, activation="gelu"), **k)), ["dy", "pre"], ["dx", "dz"]),
        "gated": (lambda **k: dq4.dq4_gated_fused(w, up, N_OUT, N_IN, 64, **dict(dict(x=x), **k)), ["x"], ["h"]),
        "gated backward": (lambda **k: dq4.dq4_gated_fused_backward(
            w, up, N_OUT, N_IN, 64, **dict(dict(dh=dy, gate_pre=g, up_pre=u), **k)),
            ["dh", "gate_pre", "up_pre"], ["dx", "dgate", "dup"]),
    }


NAMES = ["linear", "linear backward", "gated", "gated backward"]


def fresh(rows, cols):
    return torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")


def width_of(operand):
    return N_IN if operand in ("x", "dx") else N_OUT


@pytest.mark.parametrize("name", NAMES)
def test_workspace_over_a_matrix(name):
    _, w = pool_weight(51)
    _, up = pool_weight(52)
    call, ins, outs = four_calls(w, up, fresh)[name]
    for operand in ins + outs:
        space = torch.zeros(BYTES + 65536, dtype=torch.uint8, device="cuda")
        ws = space[:BYTES]
        rows = M
        inside = matrix(space, BYTES // 2, rows, width_of(operand))
        edge = matrix(space, BYTES - 256, rows, width_of(operand))   # shares its first 256 bytes
        beside = matrix(space, BYTES, rows, width_of(operand))
        for t in (inside, edge):
            with pytest.raises(ValueError, match="workspace"):
                call(**{operand: t}, workspace=ws)
        call(**{operand: beside}, workspace=ws)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("part", PARTS)
def test_workspace_over_a_weight(name, part):
    pool, w = pool_weight(53)
    _, other = pool_weight(54)
    call, _, _ = four_calls(w, other, fresh)[name]
    start = w[part].data_ptr() - pool.data_ptr()
    with pytest.raises(ValueError, match="workspace"):
        call(workspace=pool[start - BYTES + 256:start + 256])
    if name.startswith("gated"):
        call, _, _ = four_calls(other, w, fresh)[name]
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=pool[start - BYTES + 256:start + 256])
    call(workspace=pool[:BYTES])
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("part", PARTS)
def test_output_over_a_weight(name, part):
    pool, w = pool_weight(55)
    _, other = pool_weight(56)
    start = w[part].data_ptr() - pool.data_ptr()
    for first, second in ((w, other), (other, w)):
        if first is other and not name.startswith("gated"):
            continue
        call, _, outs = four_calls(first, second, fresh)[name]
        for operand in outs:
            with pytest.raises(ValueError, match=operand):
                call(**{operand: matrix(pool, start, M, width_of(operand))})
            call(**{operand: matrix(pool, 0, M, width_of(operand))})
    torch.cuda.synchronize()
