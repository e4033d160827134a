"""Device-side validation of the gated grouped call's offsets, through the C ABI of
both builds, as test_gpu_offsets.py holds the other grouped calls: the release
library writes nothing, the debug library reports FP8Q_ERR_OFFSETS and clears its
flag.  Every buffer holds more rows than any of the offsets below reaches."""

import ctypes

import pytest
import torch

from gpu_util import DEV, fq
from test_gpu_offsets import BAD, E_OFFSETS, LIB_DEBUG, OK

pytestmark = pytest.mark.gpu
G, F, K, ROWS = 3, 256, 384, 512


@pytest.fixture(scope="module")
def operands():
    f = fq()
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn((ROWS, K), generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn((G * 2 * F, K), generator=g, device=DEV) * 0.05).to(torch.bfloat16)
    wq, ws = f.quantize_weight(w)
    return (*f.quantize_act(x), wq.view(G, 2 * F, K), ws.view(G, 2 * F // 128, K // 128))


def _lib(debug):
    if not debug:
        return fq().lib
    L = ctypes.CDLL(LIB_DEBUG)
    name = "fp8q_grouped_gemm_gated"
    getattr(L, name).argtypes = getattr(fq().lib, name).argtypes
    getattr(L, name).restype = getattr(fq().lib, name).restype
    return L


def _call(L, operands, off, M_total):
    """(status, h, gate_up), both filled with NaN before."""
    aq, as_, wq, ws = operands
    d_off = torch.tensor(off, dtype=torch.int32, device=DEV)
    h = torch.full((ROWS, F), float("nan"), dtype=torch.float32, device=DEV)
    gu = torch.full((ROWS, 2 * F), float("nan"), dtype=torch.bfloat16, device=DEV)
    # (a_s has ROWS columns: M_total is less only where no tile runs)
    st = L.fp8q_grouped_gemm_gated(aq.data_ptr(), as_.data_ptr(), M_total, d_off.data_ptr(), G,
                                   wq.data_ptr(), ws.data_ptr(), F, K, 0, h.data_ptr(), 0,
                                   gu.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st, h, gu


@pytest.mark.parametrize("case", list(BAD))
def test_release_build_writes_nothing_for_invalid_offsets(operands, case):
    st, h, gu = _call(_lib(False), operands, BAD[case], 100)
    assert st == OK and torch.isnan(h).all() and torch.isnan(gu).all()


def test_debug_build_reports_invalid_offsets(operands):
    L = _lib(True)
    off = [0, 200, 200, ROWS]
    for case, bad in BAD.items():
        st, h, gu = _call(L, operands, bad, 100)
        assert st == E_OFFSETS, case
        assert torch.isnan(h).all() and torch.isnan(gu).all(), case
        # the flag has been cleared: a valid call after it, an empty expert among
        # its own, gives the release build's bits
        got, want = _call(L, operands, off, ROWS), _call(_lib(False), operands, off, ROWS)
        assert got[0] == want[0] == OK and not torch.isnan(want[1]).any()
        assert torch.equal(got[1].view(torch.int32), want[1].view(torch.int32))
        assert torch.equal(got[2].view(torch.int16), want[2].view(torch.int16))


def test_debug_flags_of_the_two_grouped_kernels_are_apart(operands):
    """An invalid gated call leaves nothing behind for the plain grouped call."""
    L = _lib(True)
    f = fq().lib.fp8q_grouped_gemm
    L.fp8q_grouped_gemm.argtypes, L.fp8q_grouped_gemm.restype = f.argtypes, f.restype
    aq, as_, wq, ws = operands
    assert _call(L, operands, BAD["decreasing"], 100)[0] == E_OFFSETS
    off = torch.tensor([0, 10, 90, ROWS], dtype=torch.int32, device=DEV)
    c = torch.empty((ROWS, 2 * F), dtype=torch.float32, device=DEV)
    assert L.fp8q_grouped_gemm(aq.data_ptr(), as_.data_ptr(), ROWS, off.data_ptr(), G,
                               wq.data_ptr(), ws.data_ptr(), 2 * F, K, c.data_ptr(), 0,
                               torch.cuda.current_stream().cuda_stream) == OK
