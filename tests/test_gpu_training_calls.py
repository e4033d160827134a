"""The training helpers' manners: allocations that dispatch modes see and deterministic
mode fills, the binding's two paths, bound calls, flags, the current stream."""

import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
M, N, F, G = 40, 256, 128, 3


class _Empties(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func in (torch.ops.aten.empty.memory_format, torch.ops.aten.empty_like.default):
            self.shapes.append(tuple(out.shape))
        return out


@pytest.fixture(scope="module")
def calls():
    """{name: (a call of stream -> outputs, the shapes it allocates)}"""
    f = fq()
    x, dy = (torch.randn(M, N, device=DEV).to(BF16) for _ in range(2))
    w, b = torch.randn(N, device=DEV), torch.randn(N, device=DEV)
    off = torch.tensor([0, 11, 11, 30], dtype=torch.int32, device=DEV)
    dh, gu = torch.randn(M, F, device=DEV).to(BF16), torch.randn(M, 2 * F, device=DEV).to(BF16)
    _, mean, rstd = f.layer_norm(x, w, b)
    T = f.expert_columns(M, G)
    work = f.layer_norm_backward_workspace(M, N)
    a, c = f.grouped_quantize_act_t(x, off), f.grouped_gated_backward(dh, gu, off)[2:]
    rows, tokens = [(M, 2 * F), (2 * F // 128, M)], [(2 * F, T), (T // 128, 2 * F)]
    return {
        "layer_norm": (lambda **k: f.layer_norm(x, w, b, 1e-5, **k), [(M, N), (M,), (M,)]),
        "layer_norm_quantized": (lambda **k: f.layer_norm_quantized(x, w, None, 1e-5, "pow2", **k),
                                 [(M, N), (N // 128, M), (M,), (M,)]),
        "layer_norm_quantized+y": (
            lambda **k: f.layer_norm_quantized(x, w, b, save_y=True, **k),
            [(M, N), (M, N), (N // 128, M), (M,), (M,)]),
        "layer_norm_backward": (lambda **k: f.layer_norm_backward(dy, x, w, mean, rstd, **k),
                                [(M, N), (N,), (N,), (work,)]),
        "layer_norm_backward-bias": (
            lambda **k: f.layer_norm_backward(dy, x, w, mean, rstd, bias=False, **k)[:2],
            [(M, N), (N,), (work,)]),
        "grouped_quantize_act_t": (lambda **k: f.grouped_quantize_act_t(x, off, **k),
                                   [(N, T), (T // 128, N)]),
        "grouped_gated_backward": (
            lambda **k: f.grouped_gated_backward(dh, gu, off, "gelu_tanh", **k), rows + tokens),
        "grouped_gated_backward tokens": (
            lambda **k: f.grouped_gated_backward(dh, gu, off, rows=False, **k)[2:], tokens),
        "grouped_gemm_rowscaled": (lambda **k: f.grouped_gemm_rowscaled(*c, *a, off, **k),
                                   [(G, 2 * F, N)]),
        "grouped_gemm_rowscaled precise": (
            lambda **k: f.grouped_gemm_rowscaled(*c, *a, off, out_dtype=BF16, precise=True, **k),
            [(G, 2 * F, N)]),
    }


NAMES = ["layer_norm", "layer_norm_quantized", "layer_norm_quantized+y", "layer_norm_backward",
         "layer_norm_backward-bias", "grouped_quantize_act_t", "grouped_gated_backward",
         "grouped_gated_backward tokens", "grouped_gemm_rowscaled",
         "grouped_gemm_rowscaled precise"]


def _written(name, out):
    """The outputs without the rows past the last expert's, which no call writes."""
    out = out if isinstance(out, tuple) else (out,)
    if name == "grouped_gated_backward":
        return (out[0][:30], out[1][:, :30], *out[2:])
    return out


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_dispatch_modes_see_the_outputs(calls, name):
    call, shapes = calls[name]
    with _Empties() as mode:
        out = call()
    assert sorted(mode.shapes) == sorted(shapes)
    assert _same(_written(name, out), _written(name, call()))


@pytest.mark.parametrize("name", NAMES)
def test_a_given_stream_and_the_current_one(calls, name):
    """Given streams take the binding's Python path."""
    call, _ = calls[name]
    want = _written(name, call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    assert _same(_written(name, call(stream=torch.cuda.current_stream())), want)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _written(name, call())
    side.synchronize()
    assert _same(got, want)
    got = _written(name, call(stream=side))
    side.synchronize()
    assert _same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(calls, name):
    call, _ = calls[name]
    want = _written(name, call())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for _ in range(3):
        for t in out if isinstance(out, tuple) else (out,):
            t.zero_()
        call()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert _same(_written(name, out), want)


def test_deterministic_mode_fills_rows_that_are_not_written(calls):
    call, _ = calls["grouped_gated_backward"]
    want = call()
    was = torch.are_deterministic_algorithms_enabled()
    fills = torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    try:
        got = call()
    finally:
        torch.use_deterministic_algorithms(was)
        torch.utils.deterministic.fill_uninitialized_memory = fills
    assert torch.isnan(got[1][:, 30:]).all() and (got[0][30:] == 255).all()
    name = "grouped_gated_backward"
    assert _same(_written(name, got), _written(name, want))


def test_bound_calls_run_again_on_the_same_buffers():
    f = fq()
    x, dy = (torch.randn(M, N, device=DEV).to(BF16) for _ in range(2))
    w = torch.randn(N, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(M, device=DEV) for _ in range(2))
    dw = torch.empty(N, device=DEV)
    work = torch.empty(f.layer_norm_backward_workspace(M, N), dtype=torch.uint8, device=DEV)
    forward = f.bind(f.fp8q_layer_norm, x, w, None, mean, rstd, y=y)
    backward = f.bind(f.fp8q_layer_norm_backward, dy, x, w, mean, rstd, dx, dw, None, work)
    p, gr = torch.randn(1000, device=DEV), torch.randn(1000, device=DEV)
    m, v = torch.zeros(1000, device=DEV), torch.zeros(1000, device=DEV)
    step = torch.ones(1, dtype=torch.int32, device=DEV)
    update = f.bind(f.fp8q_adamw, [p], [gr], [m], [v], step)
    pe, me, ve = p.clone(), m.clone(), v.clone()
    for k in range(1, 4):
        x.copy_(torch.randn(M, N, device=DEV))
        gr.copy_(torch.randn(1000, device=DEV))
        step.fill_(k)
        forward()
        backward()
        update()
        ry, rm, rr = f.layer_norm(x, w)
        assert _same((y, mean, rstd), (ry, rm, rr))
        assert _same((dx, dw), f.layer_norm_backward(dy, x, w, rm, rr, bias=False)[:2])
        f.adamw([pe], [gr], [me], [ve], step)
        assert _same((p, m, v), (pe, me, ve))


@pytest.mark.parametrize("flag", [dict(bias=np.array([1, 0])), dict(rows=np.array([1, 0])),
                                  dict(tokens=np.array([1, 0])), dict(precise=np.array([1, 0]))])
def test_flags_whose_truth_cannot_be_told(calls, flag):
    name = {"bias": "layer_norm_backward", "precise": "grouped_gemm_rowscaled"}.get(
        next(iter(flag)), "grouped_gated_backward")
    with pytest.raises(ValueError, match="ambiguous"):
        calls[name][0](**flag)


@pytest.mark.parametrize("name", ["layer_norm_quantized"])
def test_save_y_whose_truth_cannot_be_told(calls, name):
    with pytest.raises(ValueError, match="ambiguous"):
        calls[name][0](save_y=np.array([1, 0]))


def test_a_workspace_stays_taken_while_a_given_stream_uses_it(monkeypatch):
    """The workspace of a call on a stream that is behind is not handed out again."""
    f = fq()
    x = torch.randn(2000, 1024, device=DEV)
    w = torch.randn(1024, device=DEV)
    _, mean, rstd = f.layer_norm(x, w)
    entry, seen = f.fp8q_layer_norm_backward, []

    def spy(*args):
        seen.append((args[8].data_ptr(), args[8].numel()))
        entry(*args)

    monkeypatch.setattr(f, "fp8q_layer_norm_backward", spy)
    want = f.layer_norm_backward(x, x, w, mean, rstd)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)       # some 50 ms
    got = f.layer_norm_backward(x, x, w, mean, rstd, stream=side)
    taken = [torch.empty(seen[-1][1], dtype=torch.uint8, device=DEV) for _ in range(4)]
    waiting = not side.query()
    side.synchronize()
    assert waiting and seen[-1][0] not in [t.data_ptr() for t in taken]
    assert _same(got, want)


def test_a_bound_call_holds_its_lists_tensors():
    f = fq()
    lists = [[torch.randn(512, device=DEV)] for _ in range(2)] + \
        [[torch.zeros(512, device=DEV)] for _ in range(2)]
    p, others = lists[0][0], [l[0].data_ptr() for l in lists[1:]]
    run = f.bind(f.fp8q_adamw, *lists, 1)
    for l in lists:
        l.clear()
    again = [torch.empty(512, device=DEV).data_ptr() for _ in range(8)]
    assert not set(others) & set(again)
    before = p.clone()
    run()
    assert not torch.equal(p, before)
