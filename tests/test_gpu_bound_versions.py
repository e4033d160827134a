"""A bound AdamW call tells autograd of its writes as an unbound one does."""

import pytest
import torch

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu


def test_a_bound_update_is_seen_by_autograd():
    w = torch.randn(50, device=DEV, requires_grad=True)
    g, m, v = torch.ones(50, device=DEV), torch.zeros(50, device=DEV), torch.zeros(50, device=DEV)
    y = torch.empty(50, dtype=torch.bfloat16, device=DEV)
    step = torch.ones(1, dtype=torch.int32, device=DEV)
    with torch.no_grad():
        run = fq().bind(fq().fp8q_adamw, [w], [g], [m], [v], step, copies=[y])
    written = (w, m, v, y)
    for _ in range(2):
        was = [t._version for t in written]
        loss = (w * w).sum()
        run()
        assert all(t._version > k for t, k in zip(written, was)) and g._version == 0
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
