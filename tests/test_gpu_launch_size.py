"""Calls of more work than one launch takes (2^32 lanes): the first and the last
rows or columns of each launch against a call of their own."""

import pytest
import torch

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# rows of 4 to a workgroup of 256 lanes, and of one
@pytest.mark.parametrize("M,K", [(1 << 26, 1), ((1 << 26) + 7, 3), ((1 << 24) + 5, 2049)])
def test_quantize_token_i8(M, K):
    f = fq()
    x = torch.ones((M, K), dtype=torch.bfloat16, device=DEV)
    edge = (1 << 26) - 4 if K <= 2048 else (1 << 24) - 1    # first row of the second launch
    for r in (0, edge - 1, edge, M - 1):
        x[r] = torch.randn(K, generator=_gen(r), device=DEV).to(torch.bfloat16)
    q, s = f.quantize_token_i8(x)
    for r in (0, 1, edge - 1, edge, M - 1):
        q1, s1 = f.quantize_token_i8(x[r:r + 1].clone())
        assert torch.equal(q[r:r + 1], q1) and torch.equal(s[r:r + 1], s1), r
    assert int((s == 0).sum()) == 0     # every row has been written
    assert bool((s[1:edge - 1] == s[1]).all()) and bool((s[edge + 1:M - 1] == s[1]).all())


# 16 (gated: 8) weight rows to a workgroup of 512 lanes
@pytest.mark.parametrize("gated", [False, True])
def test_few_rows_int8(gated):
    f, g = fq(), _gen(1)
    cols = (1 << 23) * (8 if gated else 16) + 37
    N, M, K = cols * (2 if gated else 1), 2, 16
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    a = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    sa = torch.rand(M, generator=g, device=DEV) * 1e-2 + 1e-3
    sw = torch.rand(N, generator=g, device=DEV) * 1e-3 + 1e-4
    call = f.gemm_i8_gated if gated else f.gemm_i8
    out = call(a, sa, w, sw, out_dtype=torch.float32)
    edge = cols - 37 - (8 if gated else 16)                 # first column of the second launch
    for n0, n1 in ((0, 32), (edge - 32, edge), (edge, edge + 32), (cols - 32, cols)):
        at = torch.arange(n0, n1, device=DEV)
        r = torch.cat([at, cols + at]) if gated else at
        assert torch.equal(out[:, n0:n1], call(a, sa, w[r], sw[r], out_dtype=torch.float32)), n0


def test_few_rows_e4m3():
    f, g = fq(), _gen(2)
    F, M, K = (1 << 26) + 256, 1, 128
    w = torch.randint(0, 127, (2 * F, K), generator=g, device=DEV, dtype=torch.uint8)
    a = torch.randint(0, 127, (M, K), generator=g, device=DEV, dtype=torch.uint8)
    sa = torch.full((1, M), 1e-3, device=DEV)
    sw = torch.rand((2 * F // 128, 1), generator=g, device=DEV) * 1e-3
    h = f.gemm_gated(a, sa, w, sw, out_dtype=torch.float32)
    edge = (1 << 26) - 8                                    # first feature of the second launch
    for f0 in (0, edge // 128 * 128, edge // 128 * 128 + 128, F - 128):
        r = torch.cat([torch.arange(f0, f0 + 128), F + torch.arange(f0, f0 + 128)]).to(DEV)
        b = torch.tensor([f0 // 128, (F + f0) // 128], device=DEV)
        assert torch.equal(h[:, f0:f0 + 128],
                           f.gemm_gated(a, sa, w[r], sw[b], out_dtype=torch.float32)), f0


def test_quantize_act_refuses_what_one_launch_cannot_take():
    """16 rows of one group to a workgroup of 256 lanes: 2^28 rows are past the limit."""
    f = fq()
    M = (1 << 28) + 16
    x = torch.empty((M, 128), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((M, 128), dtype=torch.uint8, device=DEV)
    s = torch.empty((1, M), dtype=torch.float32, device=DEV)
    with pytest.raises(f.Fp8qError, match="ERR_LAUNCH"):
        f.fp8q_quantize_act(x, q, s)
    # the most that is taken
    m = M - 32
    x[:m] = 1
    s = torch.zeros((1, m), dtype=torch.float32, device=DEV)
    f.fp8q_quantize_act(x[:m], q[:m], s)
    assert bool((s == s[0, 0]).all()) and float(s[0, 0]) > 0
