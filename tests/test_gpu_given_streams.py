"""Helpers on a named stream that nothing orders against the current one: what they
allocate is no memory that pending work of the current stream still uses, and what they
return stays taken while the current stream uses it."""

import types

import pytest
import torch

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
M, N, K, F, G = 128, 256, 384, 128, 3
NAMES = ["quantize_act", "quantize_weight", "quantize_act_t", "quantize_weight_t", "gemm",
         "gemm_rowscaled", "gemm_fused", "grouped_gemm", "grouped_gemm_fused", "quantize_token_i8",
         "gemm_i8", "gemm_i8_gated", "gemm_gated", "grouped_gemm_gated", "gated_backward",
         "layer_norm", "layer_norm_quantized", "layer_norm_backward", "grouped_quantize_act_t",
         "grouped_gated_backward", "grouped_gemm_rowscaled"]


@pytest.fixture(scope="module")
def calls():
    """{name: a call of stream -> a list of outputs}"""
    f = fq()
    rand = lambda *s: torch.randn(s, device=DEV).to(BF16)   # noqa: E731
    x, w, y = rand(M, K), rand(N, K), rand(M, N)
    gamma = torch.rand(K, device=DEV) + 0.5
    off = torch.tensor([0, 50, 50, M], dtype=torch.int32, device=DEV)
    a, b = f.quantize_act(x), f.quantize_weight(w)
    bg = [torch.stack([t] * G) for t in b]
    at, yt = f.quantize_act_t(x), f.quantize_act_t(y)
    a8, b8 = f.quantize_token_i8(x), f.quantize_token_i8(w)
    dh, gu = rand(M, F), rand(M, 2 * F)
    _, mean, rstd = f.layer_norm(x, gamma)
    along, along_y = f.grouped_quantize_act_t(x, off), f.grouped_quantize_act_t(y, off)
    made = {
        "quantize_act": lambda **k: f.quantize_act(x, **k),
        "quantize_weight": lambda **k: f.quantize_weight(w, **k),
        "quantize_act_t": lambda **k: f.quantize_act_t(x, **k),
        "quantize_weight_t": lambda **k: f.quantize_weight_t(w, **k),
        "gemm": lambda **k: f.gemm(*a, *b, **k),
        "gemm_rowscaled": lambda **k: f.gemm_rowscaled(*yt, *at, **k),
        "gemm_fused": lambda **k: f.gemm_fused(x, *b, **k),
        "grouped_gemm": lambda **k: f.grouped_gemm(*a, off, *bg, **k),
        "grouped_gemm_fused": lambda **k: f.grouped_gemm_fused(x, off, *bg, **k),
        "quantize_token_i8": lambda **k: f.quantize_token_i8(x, **k),
        "gemm_i8": lambda **k: f.gemm_i8(*a8, *b8, **k),
        "gemm_i8_gated": lambda **k: f.gemm_i8_gated(*a8, *b8, **k),
        "gemm_gated": lambda **k: f.gemm_gated(*a, *b, save_gate_up=True, **k),
        "grouped_gemm_gated": lambda **k: f.grouped_gemm_gated(*a[:2], off, *bg, save_gate_up=True,
                                                               **k),
        "gated_backward": lambda **k: f.gated_backward(dh, gu, **k),
        "layer_norm": lambda **k: f.layer_norm(x, gamma, **k),
        "layer_norm_quantized": lambda **k: f.layer_norm_quantized(x, gamma, save_y=True, **k),
        "layer_norm_backward": lambda **k: f.layer_norm_backward(x, x, gamma, mean, rstd, **k),
        "grouped_quantize_act_t": lambda **k: f.grouped_quantize_act_t(x, off, **k),
        "grouped_gated_backward": lambda **k: f.grouped_gated_backward(dh, gu, off, **k),
        "grouped_gemm_rowscaled": lambda **k: f.grouped_gemm_rowscaled(*along_y, *along, off, **k),
    }
    assert sorted(made) == sorted(NAMES)

    def outputs(call):
        def run(**k):
            out = call(**k)
            return list(out) if isinstance(out, tuple) else [out]
        return run
    return {n: outputs(c) for n, c in made.items()}


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


def _delay():
    torch.cuda._sleep(100_000_000)       # some 50 ms


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_writes_is_not_taken(calls, name):
    """Blocks of the outputs' sizes, freed while the fills of them are still pending."""
    call = calls[name]
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    _delay()
    junk = [torch.empty_like(t) for t in want]
    for t in junk:
        t.view(torch.uint8).fill_(0x5A)
    del junk, t
    got = call(stream=side)
    waiting = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert waiting and _same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_stay_taken_while_the_current_stream_reads_them(calls, name):
    """Outputs dropped while copies of them are pending: the next call on that stream
    writes elsewhere."""
    call = calls[name]
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    out = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _delay()
    copies = [t.clone() for t in out]
    del out
    again = call(stream=side)
    with torch.cuda.stream(side):
        for t in again:
            t.view(torch.uint8).fill_(0x5A)
    waiting = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert waiting and _same(copies, want)


def test_a_workspace_in_use_on_the_current_stream_is_not_taken(monkeypatch):
    """Two backward passes of one shape at once, on the current stream and on another."""
    f = fq()
    x = torch.randn(2000, 1024, device=DEV)
    w = torch.randn(1024, device=DEV)
    _, mean, rstd = f.layer_norm(x, w)
    want = f.layer_norm_backward(x, x, w, mean, rstd)
    entry, seen = f.fp8q_layer_norm_backward, []

    def spy(*args):
        seen.append((args[8].data_ptr(), args[8].numel()))
        entry(*args)

    monkeypatch.setattr(f, "fp8q_layer_norm_backward", spy)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    _delay()
    one = f.layer_norm_backward(x, x, w, mean, rstd, stream=torch.cuda.current_stream())
    two = f.layer_norm_backward(x, x, w, mean, rstd, stream=side)
    waiting = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    (a, n), (b, _) = seen
    assert waiting and (a + n <= b or b + n <= a)
    assert _same(one, want) and _same(two, want)


@pytest.mark.parametrize("name", ["gemm", "layer_norm_backward"])
def test_any_object_that_has_a_stream(calls, name):
    call = calls[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert _same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_captured_beside_the_capturing_stream(calls, name):
    """A graph whose call runs on a stream of its own, joined to the captured one."""
    call = calls[name]
    want = call()
    side = torch.cuda.Stream()
    call(stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in out:
            t.zero_()
        call()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert _same(out, want)
