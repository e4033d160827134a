"""Training calls on views that begin where only 4-byte alignment is left (scales, weights,
statistics, offsets, device scalars), in threads of their own, and captured with more
tensors than one launch describes."""

import threading

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq
from test_gpu_adamw import Tensors

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _shifted(t, by=1):
    """A contiguous copy of t that begins `by` elements into its storage."""
    room = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    room.fill_(7)
    room[by:] = t.reshape(-1)
    return room[by:].view(t.shape)


def _same(a, b):
    return all(x.shape == y.shape and
               (x.numel() == 0 or torch.equal(x.contiguous().view(torch.uint8),
                                              y.contiguous().view(torch.uint8)))
               for x, y in zip(a, b))


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("M,N", [(5, 77), (33, 128), (7, 1024), (3, 1001), (6, 7168), (2, 9000)])
def test_layer_norm(M, N, by):
    f = fq()
    x, dy = (torch.randn((M, N), device=DEV).to(BF16) for _ in range(2))
    w, b = torch.rand(N, device=DEV) + 0.5, torch.randn(N, device=DEV)
    y, mean, rstd = f.layer_norm(x, w, b)
    want = f.layer_norm_backward(dy, x, w, mean, rstd)
    got = f.layer_norm(x, _shifted(w, by), _shifted(b, by))
    assert _same(got, (y, mean, rstd))
    new = lambda n: _shifted(torch.zeros(n, device=DEV), by)   # noqa: E731
    mean2, rstd2, dw, db = new(M), new(M), new(N), new(N)
    y2, dx = torch.empty_like(y), torch.empty_like(x)
    q = s = None
    if N % 128 == 0:
        q, s = torch.empty((M, N), dtype=torch.uint8, device=DEV), new(N // 128 * M).view(N // 128, M)
    f.fp8q_layer_norm(x, _shifted(w, by), _shifted(b, by), mean2, rstd2, y2, q, s)
    assert _same((y2, mean2, rstd2), (y, mean, rstd))
    if q is not None:
        assert _same((q, s), f.layer_norm_quantized(x, w, b)[:2])
    work = torch.empty(f.layer_norm_backward_workspace(M, N), dtype=torch.uint8, device=DEV)
    f.fp8q_layer_norm_backward(dy, x, _shifted(w, by), mean2, rstd2, dx, dw, db, work)
    assert _same((dx, dw, db), want)


@pytest.mark.parametrize("by", [1, 3])
def test_experts(by):
    f = fq()
    M, K, F, counts = 700, 384, 256, [0, 5, 300, 0, 128, 267]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    x = torch.randn((M, K), device=DEV).to(BF16)
    dh, gu = torch.randn((M, F), device=DEV).to(BF16), torch.randn((M, 2 * F), device=DEV).to(BF16)
    at, gt = f.grouped_quantize_act_t(x, off), f.grouped_gated_backward(dh, gu, off)
    want = f.grouped_gemm_rowscaled(*gt[2:], *at, off)
    off2 = _shifted(off, by)
    assert _same(f.grouped_quantize_act_t(x, off2), at)
    assert _same(f.grouped_gated_backward(dh, gu, off2), gt)
    for precise in (False, True):
        w = f.grouped_gemm_rowscaled(gt[2], _shifted(gt[3], by), at[0], _shifted(at[1], by), off2,
                                     precise=precise)
        if not precise:
            assert _same([w], [want])
        else:
            assert _same([w], [f.grouped_gemm_rowscaled(*gt[2:], *at, off, precise=True)])
    q_t, s_t = torch.empty_like(at[0]), _shifted(torch.zeros_like(at[1]), by)
    f.fp8q_grouped_quantize_act_t(x, off2, q_t, s_t)
    assert _same((q_t, s_t), at)


def test_adamw_scales_and_scalars():
    a, b = (Tensors([1000, 129], True, "bf16", seed=4) for _ in range(2))
    b.msd, b.vsd = [_shifted(t) for t in b.msd], [_shifted(t, 3) for t in b.vsd]
    scalar = lambda v, dt: _shifted(torch.tensor([v], dtype=dt, device=DEV))   # noqa: E731
    lr = float(np.float32(1e-3))
    for step in (1, 2, 3):
        a.call(step, lr=lr, scale=torch.tensor([0.3], device=DEV))
        b.call(scalar(step, torch.int32), lr=scalar(lr, torch.float32), scale=scalar(0.3, torch.float32))
        assert _same(a.state(), b.state())


@pytest.mark.parametrize("eight", [False, True])
def test_adamw_of_many_tensors_captured(eight):
    """150 tensors: three launches with the most arguments one takes, replayed with eager
    steps of a second set between."""
    sizes = [(37 * i) % 5000 for i in range(150)]
    a, b = (Tensors(sizes, eight, "f32", seed=6) for _ in range(2))
    step = torch.ones(1, dtype=torch.int32, device=DEV)
    for t in (a, b):
        t.call(step)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(step)
    for k in range(2, 6):
        step.fill_(k)
        for x, y in zip(a.gd, b.gd):
            x.normal_()
            y.copy_(x)
        b.call(k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert _same(a.state(), b.state())


def test_calls_from_two_threads():
    """Each thread on a stream of its own."""
    f = fq()
    x = torch.randn((300, 1024), device=DEV).to(BF16)
    w = torch.rand(1024, device=DEV) + 0.5
    y, mean, rstd = f.layer_norm(x, w)
    want = (y, *f.layer_norm_backward(x, x, w, mean, rstd))
    a = [Tensors([3000, 77], True, "f32", seed=5) for _ in range(3)]
    for k in range(1, 21):
        a[2].call(k)
    torch.cuda.synchronize()
    bad = []

    def work(t):
        with torch.cuda.stream(torch.cuda.Stream()):
            for k in range(1, 21):
                t.call(k)
                y2, m2, r2 = f.layer_norm(x, w)
                if not _same((y2, *f.layer_norm_backward(x, x, w, m2, r2)), want):
                    bad.append(k)
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(t,)) for t in a[:2]]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and _same(a[0].state(), a[2].state()) and _same(a[1].state(), a[2].state())
