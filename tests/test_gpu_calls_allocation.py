"""The feed-forward helpers' allocations are seen by torch's dispatch modes and
filled by its deterministic mode, as those of the other helpers are."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class _Empties(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.shapes.append(tuple(out.shape))
        return out


@pytest.fixture(scope="module")
def calls():
    """{name: (a call, its outputs' shapes)}"""
    f = fq()
    M, K, F = 40, 256, 128
    x, w = torch.randn(M, K, device=DEV).to(BF16), torch.randn(2 * F, K, device=DEV).to(BF16)
    a8, w8 = f.quantize_token_i8(x), f.quantize_token_i8(w)
    a, wq = f.quantize_act(x), f.quantize_weight(w)
    off = torch.tensor([0, 11, 30], dtype=torch.int32, device=DEV)
    w3 = [torch.stack([t, t]) for t in wq]
    dh, gu = torch.randn(M, F, device=DEV).to(BF16), torch.randn(M, 2 * F, device=DEV).to(BF16)
    return {
        "quantize_act": (lambda: f.quantize_act(x), [(M, K), (K // 128, M)]),
        "quantize_token_i8": (lambda: f.quantize_token_i8(x), [(M, K), (M,)]),
        "gemm_i8": (lambda: f.gemm_i8(*a8, *w8), [(M, 2 * F)]),
        "gemm_i8_gated": (lambda: f.gemm_i8_gated(*a8, *w8), [(M, F)]),
        "gemm_gated": (lambda: f.gemm_gated(*a, *wq, save_gate_up=True), [(M, F), (M, 2 * F)]),
        "grouped_gemm_gated": (lambda: f.grouped_gemm_gated(*a, off, *w3), [(M, F)]),
        "gated_backward": (lambda: f.gated_backward(dh, gu),
                           [(M, 2 * F), (2 * F // 128, M), (2 * F, 128), (1, 2 * F)]),
    }


NAMES = ["quantize_act", "quantize_token_i8", "gemm_i8", "gemm_i8_gated", "gemm_gated",
         "grouped_gemm_gated", "gated_backward"]


def _same(a, b):
    a, b = [t if isinstance(t, tuple) else (t,) for t in (a, b)]
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_dispatch_modes_see_the_outputs(calls, name):
    call, shapes = calls[name]
    with _Empties() as mode:
        out = call()
    assert mode.shapes == shapes
    if name != "grouped_gemm_gated":      # (whose rows past the offsets are not written)
        assert _same(out, call())


def test_deterministic_mode_fills_rows_that_are_not_written(calls):
    call, _ = calls["grouped_gemm_gated"]
    want = call()
    was = torch.are_deterministic_algorithms_enabled()
    fills = torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    try:
        h = call()
    finally:
        torch.use_deterministic_algorithms(was)
        torch.utils.deterministic.fill_uninitialized_memory = fills
    assert torch.isnan(h[30:]).all()
    assert _same(h[:30], want[:30])
