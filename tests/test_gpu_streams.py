"""Calls with an explicit stream: what they allocate belongs to that stream.

The allocator gives a block back to the stream that it was allocated on.  A
result or scratch buffer of the current stream's, used on another one, may be
in use by earlier work of the current stream, and may be handed to later work
of it while the call still runs.  Both orders are made to happen here, by a
stream that is held up (some 50 ms of waiting in a kernel); bits have to be
those of a call on the current stream.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import mixed_precision_dense_02_gb300 as mma
from mixed_precision_dense_02_gb300 import binding

pytestmark = pytest.mark.gpu

HELD = 100_000_000  # clocks


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


def rnd(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def calls():
    """The calls, each with its inputs: f(stream=...) gives its results."""
    m, n, k = 700, 512, 640
    x, h, dy, r = (rnd(i, m, k) for i in range(4))
    w = rnd(5, k)
    a, sa = mma.quantize_f8(x)
    b, sb = mma.quantize_f8(rnd(6, n, k), block_rows=128)
    at = torch.tensor([0, 300, 300, m], dtype=torch.int32, device="cuda")
    e = rnd(7, 3, n, k)
    e8, se = zip(*(mma.quantize_f8(v, block_rows=128) for v in e))
    e8 = torch.stack([v.view(torch.uint8) for v in e8]).view(a.dtype)
    se, y = torch.stack(se), rnd(8, m, n)
    i8 = torch.arange(m * k, device="cuda").remainder(255).sub(127).to(torch.int8).view(m, k)
    xb = x[:512].reshape(8, 64, k).contiguous()
    return {
        "norm": lambda **s: mma.rmsnorm_f8(x, w, r, y=True, **s),
        "norm backward": lambda **s: mma.rmsnorm_backward(dy, h, w, r, **s),
        "quantise": lambda **s: mma.quantize_f8(x, transpose=True, **s),
        "f8": lambda **s: mma.gemm_f8(a, sa, b, sb, **s),
        "grouped": lambda **s: mma.gemm_grouped(x, e, at, **s),
        "grouped gradient": lambda **s: mma.gemm_grouped_wgrad(y, x, at, **s),
        "grouped f8": lambda **s: mma.gemm_grouped_f8(a, sa, e8, se, at, **s),
        "gemm": lambda **s: mma.gemm(x, e[0], **s),
        "gemm_i8_ex": lambda **s: mma.gemm_i8_ex(i8, i8[:n], **s),
        "gemm_batched": lambda **s: mma.gemm_batched(xb, xb, **s),
    }


def tensors(out):
    return [t.view(torch.uint8) if t.dtype.itemsize == 1 else t
            for t in (out if isinstance(out, tuple) else (out,))]


def same(got, want):
    return all(bool((g == w).all()) for g, w in zip(tensors(got), want))


NAMES = ["norm", "norm backward", "quantise", "f8", "grouped", "grouped gradient", "grouped f8",
         "gemm", "gemm_i8_ex", "gemm_batched"]


@pytest.mark.parametrize("name", NAMES)
def test_results_are_not_in_use_by_the_current_stream(name):
    """Blocks freed on the current stream whose last use is still to come."""
    f = calls()[name]
    want = [t.clone() for t in tensors(f())]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = [t.untyped_storage().nbytes() for t in want] + [binding.load().mma_rmsnorm_backward_workspace(700, 640)]
    old = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(3)]
    torch.cuda._sleep(HELD)
    for t in old:
        t.fill_(0x55)
    del old, t
    got = f(stream=other)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("handle", [False, True])
def test_scratch_is_not_handed_out_while_the_call_runs(name, handle):
    """Allocations on the current stream while the call waits on the other."""
    f = calls()[name]
    want = [t.clone() for t in tensors(f())]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(HELD)
    got = f(stream=other.cuda_stream if handle else other)
    need = binding.load().mma_rmsnorm_backward_workspace(700, 640)
    new = [torch.full((s,), 0x55, dtype=torch.uint8, device="cuda")
           for s in (need, need // 2, 4096) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((t == 0x55).all()) for t in new)
    assert same(got, want)


def test_default_stream_by_handle():
    f = calls()["norm backward"]
    want = [t.clone() for t in tensors(f())]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = f(stream=0)
    torch.cuda.synchronize()
    assert same(got, want)
