"""Weight gradients by expert over the most columns a call takes (2^24): the last tokens of
a tile's last row, 2^32 bytes behind its first row's."""

import pytest
import torch

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts", [1024, 1])
def test_last_tokens_of_the_longest_operands(experts):
    """All tokens are the first expert's.  1024 experts are enough tiles for those of 256
    rows, one expert takes those of 128.  Codes are zero (their products exact) but in
    the last group, so that every row's last tokens count."""
    T, N, K = 1 << 24, 512, 256
    a, b = (torch.zeros((n, T), dtype=torch.uint8, device=DEV) for n in (N, K))
    one = 0x38                                   # 1.0 in E4M3
    a[:, -128:] = one
    b[:, -128:] = one
    a_s, b_s = (torch.ones((T // 128, n), device=DEV) for n in (N, K))
    off = torch.full((experts + 1,), T, dtype=torch.int32, device=DEV)
    off[0] = 0
    c = fq().grouped_gemm_rowscaled(a, a_s, b, b_s, off)
    assert bool((c[0] == 128).all())
    assert not c[1:].any()
