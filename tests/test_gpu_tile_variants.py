"""Every kernel that the choice can take, each at shapes that test_tile_choice.py
shows it to be taken for: the largest sums of int8 codes, and long K with the rings
many rounds in and a part of a chunk at the end.  References and tolerances as in
test_gpu_feed_forward_large."""

import numpy as np
import pytest
import torch

import test_gpu_feed_forward as small
import test_gpu_feed_forward_large as large
import tile_shapes as ts
from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu
U = large.U


def _ids(shapes):
    return [f"{tile}-{'x'.join(map(str, s))}" for tile, s in shapes.items()]


@pytest.mark.parametrize("M,N", ts.I8_LARGEST_SUM.values(), ids=_ids(ts.I8_LARGEST_SUM))
def test_gemm_i8_largest_sum(M, N):
    """Codes of -128 and 127; rows and weight rows of -128 alone: 2^31 - 2^18, still an int32."""
    K, g = ts.I8_LARGEST_SUM_K, large._gen(M)
    a, w = [127 - torch.randint(0, 2, (n, K), generator=g, device=DEV, dtype=torch.int8)
            for n in (M, N)]
    a, w = [torch.where(t == 126, -128, t) for t in (a, w)]
    for t, n in ((a, M), (w, N)):
        t[[0, n // 2, n - 1]] = -128
    sa, sw = large._pos(g, M), large._pos(g, N)
    c = fq().gemm_i8(a, sa, w, sw)
    at = torch.cat([torch.arange(0, 40), torch.arange(M // 2 - 20, M // 2 + 20),
                    torch.arange(M - 40, M)]).unique().to(DEV)
    p = a[at].double() @ w.double().t()
    assert float(p.max()) == 2.0 ** 31 - 2.0 ** 18
    assert large._close(c[at], p * sa[at].double()[:, None] * sw.double(), 4 * U)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", ts.I8_LONG_K.values(), ids=_ids(ts.I8_LONG_K))
def test_gemm_i8_long_k(M, N, K, out):
    large.test_gemm_i8_tiles(M, N, K, True, out)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", ts.I8_GATED_LONG_K.values(), ids=_ids(ts.I8_GATED_LONG_K))
def test_gemm_i8_gated_long_k(M, F, K, act):
    large.test_gemm_i8_gated_tiles(M, F, K, act)


def test_gemm_gated_few_rows_long_k():
    """(Its order of the chunks is its own: held to the bound.)"""
    M, F, K = ts.GATED_LONG_K[0]
    qa, sa, qw, sw = small._e4m3_operands(np.random.default_rng(M), M, 2 * F, K, outliers=True)
    h, gu = fq().gemm_gated(*[small._u8(t) for t in (qa, sa, qw, sw)], out_dtype=torch.float32,
                            save_gate_up=True)
    small._check_gated("silu", h, gu, qa, sa, qw, sw)


@pytest.mark.parametrize("M", [3, 300])
def test_gemm_gated_weights_past_4_gib(M):
    """Blocks of features of a large layer against the same features alone, every
    output: the kernel for few rows bit for bit; the tiles' sums bit for bit those
    of fp8q_gemm."""
    f, g, F, K = fq(), large._gen(5), 40960, 57344
    a, sa, w, sw = large._gated_inputs(g, M, F, K)
    h, gu = f.gemm_gated(a, sa, w, sw, out_dtype=torch.float32, save_gate_up=True)
    for f0 in (0, 37376, 37504, F - 128):     # (37449: the weight row at 2^31 bytes)
        r = torch.cat([torch.arange(f0, f0 + 128), F + torch.arange(f0, f0 + 128)]).to(DEV)
        b = torch.tensor([f0 // 128, (F + f0) // 128], device=DEV)
        alone = a, sa, w[r].contiguous(), sw[b].contiguous()
        part = torch.cat([gu[:, f0:f0 + 128], gu[:, F + f0:F + f0 + 128]], dim=1)
        if M <= 16:
            h1, gu1 = f.gemm_gated(*alone, out_dtype=torch.float32, save_gate_up=True)
            assert torch.equal(h[:, f0:f0 + 128], h1) and torch.equal(part, gu1)
        else:
            y = f.gemm(*alone)
            assert torch.equal(part, y.to(torch.bfloat16))
            large._check_h(h[:, f0:f0 + 128], y, 128, "silu")


TILES = {t: s for t, s in ts.GATED_LONG_K.items() if t}


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", TILES.values(), ids=_ids(TILES))
def test_gemm_gated_long_k(M, F, K, act):
    large.test_gemm_gated_tiles_form_the_gemms_sums(M, F, K, act)
