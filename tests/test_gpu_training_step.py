"""Layer norm, experts, their weight gradients and AdamW as a training step uses
them together: the example's ExpertLayer."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward_experts", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def _rows(seed, M, hidden):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((M, hidden)).astype(np.float32)).to(DEV).to(BF16)


def _state(layer):
    return [*layer.w, *layer.copies, *layer.norm, layer.step,
            *[t for ts in (*layer.moments, *layer.norm_moments) for t in ts]]


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


def _reference(layer, x, counts, dy):
    """Outputs and gradients in float64 on the CPU, by automatic differentiation of the
    formulas with no rounding between the given BF16 inputs and the results."""
    leaf = lambda t: t.detach().double().cpu().requires_grad_()   # noqa: E731
    xr, w1, w2 = leaf(x), leaf(layer.copies[0]), leaf(layer.copies[1])
    g, b = leaf(layer.norm[0]), leaf(layer.norm[1])
    n = torch.nn.functional.layer_norm(xr, (x.shape[1],), g, b, 1e-5)
    ys, lo = [], 0
    for e, c in enumerate(counts):
        gate, up = (n[lo:lo + c] @ w1[e].T).chunk(2, dim=1)
        ys.append((torch.nn.functional.silu(gate) * up) @ w2[e].T)
        lo += c
    y = torch.cat(ys)
    y.backward(dy.double().cpu())
    return y.detach(), xr.grad, [w1.grad, w2.grad], [g.grad, b.grad]


@pytest.mark.parametrize("counts", [[100, 0, 29, 127], [1, 0, 0, 0], [0, 3, 300, 129], [128, 128, 0, 1]])
def test_gradients_of_the_block(example, counts):
    """Against float64, as norms.  A value in [1, 2) times a power of two has a code off by
    2^-4 at most, 2^-4 / sqrt(3) = 0.036 in the root mean square, relative to a value whose
    root mean square is 1.53: r = 0.024.  Errors of independent products add up as the
    products' own random walk does, so a product of two coded operands is off by 1.4 r of
    its norm.  Gate and up: 1.4 r.  h: of both factors', silu's slope up to 1.1 and its
    value at least half of its argument's on the side that counts, 3 r.  y: h's, its codes'
    and the weights', 3.4 r.  dh: 1.4 r; dY: dh's and 3 r of gate and up's, 3.3 r, with its
    codes' 3.5 r; dw1 and dn one more, 3.7 r; dw2 h's 3 r and two codes', 3.4 r.  The norm's
    gradients are linear in dn.  At most 0.09; twice that is allowed."""
    hidden, ffn, M = 256, 128, sum(counts)
    layer = example.ExpertLayer(hidden, ffn, 4, 5)
    rng = np.random.default_rng(8)
    for t, mean in zip(layer.norm, (1.0, 0.0)):
        t.copy_(torch.from_numpy(mean + 0.2 * rng.standard_normal(hidden)))
    x, dy = _rows(6, M, hidden), _rows(7, M, hidden)
    y = layer.forward(x, _offsets(counts))
    dx, dw, dnorm = layer.backward(dy)
    ry, rdx, rdw, rdnorm = _reference(layer, x, counts, dy)
    for got, ref in ((y, ry), (dx, rdx), *zip(dw, rdw), *zip(dnorm, rdnorm)):
        got = got.double().cpu()
        assert got.shape == ref.shape
        assert float((got - ref).norm()) <= 0.18 * float(ref.norm())
    for e, c in enumerate(counts):
        if c == 0:
            assert not dw[0][e].any() and not dw[1][e].any()


def _step(layer, x, off, dy, lr=1e-3):
    y = layer.forward(x, off)
    dx, dw, dnorm = layer.backward(dy)
    layer.update(dw, dnorm, lr)
    return [y, dx, *dw, *dnorm]


ROUTES = [[100, 0, 29, 127], [0, 0, 0, 256], [64, 64, 64, 64], [1, 255, 0, 0], [85, 85, 85, 1]]


def test_captured_step_replays_the_eager_steps(example):
    """Five steps, each with rows, routing and gradient of its own, replayed with eager
    steps of a second layer between: the same outputs and the same state, bit for bit."""
    hidden, ffn, M = 256, 128, 256
    layer, eager = (example.ExpertLayer(hidden, ffn, 4, 9) for _ in range(2))
    x, dy, off = _rows(1, M, hidden), _rows(2, M, hidden), _offsets(ROUTES[0])
    for l in (layer, eager):
        _step(l, x, off, dy)                  # (loads the kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(layer, x, off, dy)
    for k, counts in enumerate(ROUTES):
        xk, dyk, offk = _rows(10 + k, M, hidden), _rows(20 + k, M, hidden), _offsets(counts)
        want = _step(eager, xk, offk, dyk)
        torch.cuda.synchronize()
        for t, v in ((x, xk), (dy, dyk), (off, offk)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, want), k
        assert _same(_state(layer), _state(eager)), k


def test_two_graphs_in_turn(example):
    """Two captured steps of two layers share nothing: replays in turn on two streams."""
    M, hidden, ffn = 256, 256, 128
    x, dy = _rows(1, M, hidden), _rows(2, M, hidden)
    offs = [_offsets(ROUTES[0]), _offsets(ROUTES[3])]
    layers = [example.ExpertLayer(hidden, ffn, 4, seed) for seed in (1, 2)]
    twins = [example.ExpertLayer(hidden, ffn, 4, seed) for seed in (1, 2)]
    graphs = []
    for l, t, off in zip(layers, twins, offs):
        for z in (l, t):
            _step(z, x, off, dy)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            _step(l, x, off, dy)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _ in range(3):
        for t, off in zip(twins, offs):
            _step(t, x, off, dy)
    torch.cuda.synchronize()
    for l, t in zip(layers, twins):
        assert _same(_state(l), _state(t))


def test_steps_on_two_streams_at_once(example):
    hidden, ffn, M = 512, 256, 256
    x, dy = _rows(3, M, hidden), _rows(4, M, hidden)
    off = _offsets(ROUTES[0])
    a, b, ta, tb = (example.ExpertLayer(hidden, ffn, 4, s) for s in (1, 2, 1, 2))
    for _ in range(3):
        for t in (ta, tb):
            _step(t, x, off, dy)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for l, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                _step(l, x, off, dy)
    torch.cuda.synchronize()
    assert _same(_state(a), _state(ta)) and _same(_state(b), _state(tb))


def test_example_trains_experts(example):
    """Its captured training runs, and its state stays finite."""
    target, layer = (example.ExpertLayer(256, 128, 4, s) for s in (20, 21))
    first, last = example.train_experts(layer, target, _rows(5, 256, 256), _offsets(ROUTES[0]), 6,
                                        1e-3)
    assert np.isfinite(first) and np.isfinite(last)
    assert int(layer.step) == 6
    assert all(bool(torch.isfinite(t.float()).all()) for t in (*layer.w, *layer.norm))
    assert _same(layer.copies, [w.to(BF16) for w in layer.w])
