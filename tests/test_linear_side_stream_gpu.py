"""Memory of calls on a stream other than torch's current one.

What the binding allocates for a call with stream= (a workspace, outputs that
are not given) is written by kernels on that stream, which does not wait for
the current stream.  A block that was freed on the current stream may still be
read or written by work queued there, and torch's caching allocator gives such
a block to the next allocation on the current stream at once; so these tensors
come from the given stream's own memory, in whose order their kernels run.
"""
from __future__ import annotations

import pytest

import block_wise_bit_amd as dq4
from block_wise_bit_amd import inputs

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

N_OUT, N_IN, M = 1024, 2048, 200


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from libs import ensure_hip_library
    ensure_hip_library()


def make_weight(seed):
    x = inputs.make_inputs(N_OUT * N_IN, 64, "nf4", 0.03, seed=seed, n_rows=N_OUT, n_cols=N_IN)
    return dict(dq4.to_device(x), offset=float(x.offset))


def calls():
    """{name: a call of every entry point that allocates, taking stream=}."""
    w, up = make_weight(31), make_weight(32)
    sizes = dict(n_out=N_OUT, n_in=N_IN, blocksize=64)
    x = torch.ones((M, N_IN), dtype=torch.bfloat16, device="cuda")
    dy = torch.ones((M, N_OUT), dtype=torch.bfloat16, device="cuda")
    src1 = torch.ones((N_OUT, 64), dtype=torch.float32, device="cuda")
    a = torch.ones((16, N_IN), dtype=torch.float16, device="cuda")
    cb = torch.ones((N_OUT, N_IN), dtype=torch.int8, device="cuda")
    scb = torch.ones(N_OUT, device="cuda")
    cols = torch.arange(8, device="cuda")
    shape = dict(n_rows=N_OUT, n_cols=N_IN, blocksize=64, src1=src1)
    n = N_OUT * N_IN
    return {
        "linear": lambda **k: dq4.dq4_linear_fused(**w, **sizes, x=x, **k),
        "linear backward": lambda **k: dq4.dq4_linear_fused_backward(**w, **sizes, dy=dy, pre=dy, activation="silu",
                                                                     bias_grad=True, **k),
        "gated": lambda **k: dq4.dq4_gated_fused(w, up, N_OUT, N_IN, 64, x, **k),
        "gated backward": lambda **k: dq4.dq4_gated_fused_backward(w, up, N_OUT, N_IN, 64, dy, dy, dy, **k),
        "dequant": lambda **k: dq4.dq4_nested_dequant(**w, n=n, blocksize=64, **k),
        "dequant rows": lambda **k: dq4.dq4_nested_dequant_rows(**w, n_rows=N_OUT, n_cols=N_IN, r0=3, rows=100,
                                                                blocksize=64, **k),
        "unfused": lambda **k: dq4.dq4_nested_dequant_unfused(**w, n=n, blocksize=64, **k),
        "unfused noalloc": lambda **k: dq4.dq4_nested_dequant_unfused_noalloc(**w, n=n, blocksize=64, **k),
        "out_prod rows": lambda **k: dq4.dq4_out_prod_rows(**w, **shape, **k),
        "out_prod": lambda **k: dq4.dq4_out_prod_fused(**w, **shape, **k),
        "dequant linear": lambda **k: dq4.dq4_dequant_linear(**w, **sizes, x=x, **k),
        "int8 prep": lambda **k: dq4.dq4_int8_prep(a, cb, scb, cols, **k),
        "memory twin": lambda **k: dq4.dq4_memory_twin_f16(w["packed"], n, **k),
    }


NAMES = ["linear", "linear backward", "gated", "gated backward", "dequant", "dequant rows", "unfused",
         "unfused noalloc", "out_prod rows", "out_prod", "dequant linear", "int8 prep", "memory twin"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_come_from_the_given_stream(name, monkeypatch):
    call = calls()[name]
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
    assert [s for s, n in made if n], f"{name} allocated nothing"
    assert all(s == side.cuda_stream for s, n in made if n), f"{name} took the current stream's memory"
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))   # bits: the twin's are no numbers


@pytest.mark.parametrize("name", ["linear", "gated", "linear backward"])
def test_workspace_is_not_one_still_read_on_the_current_stream(name, monkeypatch):
    """A call on the current stream drops its workspace
    while its kernels are queued; a call on another stream must not get it."""
    call = calls()[name]
    side = torch.cuda.Stream()
    call()
    call(stream=side)
    torch.cuda.synchronize()
    blocks = []
    empty = torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        blocks.append((t.data_ptr(), t.numel() * t.element_size()))
        return t
    monkeypatch.setattr(torch, "empty", spy)
    keep = call()
    first, blocks[:] = list(blocks), []
    other = call(stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert first and blocks
    for p, n in blocks:
        for q, k in first:
            assert p >= q + k or q >= p + n, f"{name}: a block of the first call was handed to the second"
    del keep, other


def test_outputs_of_a_side_stream_outlive_their_use_on_the_current_one(monkeypatch):
    """A returned tensor is marked as used on the caller's current stream: when
    it is freed, the given stream's next call does not get its memory before
    the current stream's work queued so far is done."""
    call = calls()["dequant"]
    side = torch.cuda.Stream()
    marked = []
    record = torch.Tensor.record_stream

    def spy(t, stream):
        marked.append((t.data_ptr(), stream.cuda_stream))
        return record(t, stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", spy)
    y = call(stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert (y.data_ptr(), torch.cuda.current_stream().cuda_stream) in marked


@pytest.mark.parametrize("name", ["linear", "linear backward", "gated", "gated backward", "out_prod"])
def test_captured_on_a_forked_stream(name):
    """A graph whose capture forks to another stream for the call and joins it
    again; replayed with eager calls of the same kind in between."""
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call()
    call(stream=side)
    torch.cuda.synchronize()
    want = want if isinstance(want, tuple) else (want,)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = call(stream=side)
        main.wait_stream(side)
    got = got if isinstance(got, tuple) else (got,)
    for _ in range(3):
        for t in got:
            if t.data_ptr() not in [w.data_ptr() for w in want]:
                t.zero_()
        call()
        g.replay()
        call(stream=side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


class OtherDevice:
    """A stream of a device that is not the tensors'."""
    device = torch.device("cuda", 1)
    cuda_stream = 0


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(name):
    call = calls()[name]
    assert torch.cuda.current_device() == 0
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(stream=OtherDevice())
    torch.cuda.synchronize()


def test_a_stream_of_another_device_is_refused_with_everything_given():
    w = make_weight(33)
    x = torch.ones((1, N_IN), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((1, N_OUT), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        dq4.dq4_linear_fused(**w, n_out=N_OUT, n_in=N_IN, blocksize=64, x=x, y=y, stream=OtherDevice())
    out = torch.empty(N_OUT * N_IN, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        dq4.dq4_nested_dequant(**w, n=N_OUT * N_IN, blocksize=64, out=out, stream=OtherDevice())
