"""Flags of the feed-forward helpers whose truth cannot be told: Python's own error."""

import numpy as np
import pytest
import torch

fq = pytest.importorskip("fine_grained_block_fp8q_amd")
BF16 = torch.bfloat16


@pytest.mark.parametrize("flag", ["rows", "tokens"])
def test_gated_backward(flag):
    with pytest.raises(ValueError, match="ambiguous"):
        fq.gated_backward(torch.empty((4, 128), dtype=BF16), torch.empty((4, 256), dtype=BF16),
                          **{flag: np.array([1, 0])})


@pytest.mark.gpu
def test_gemm_gated():
    z = lambda s, d: torch.zeros(s, dtype=d, device="cuda")   # noqa: E731
    with pytest.raises(ValueError, match="ambiguous"):
        fq.gemm_gated(z((4, 128), torch.uint8), z((1, 4), torch.float32),
                      z((256, 128), torch.uint8), z((2, 1), torch.float32),
                      save_gate_up=np.array([1, 0]))
