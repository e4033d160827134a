"""AdamW's factors where some scalars are on the device: formed in 64 bits and rounded
once, so every combination gives the same bits at every step."""

import numpy as np
import pytest
import torch

from gpu_util import DEV
from test_gpu_adamw import Tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eight", [False, True])
def test_rate_on_the_device_and_step_on_the_host(eight):
    """Steps 1 to 200 (1 - 0.9^t is not yet 1) in each of the four combinations; over
    them 1 / (1 - 0.9^t) rounded to FP32 before its product with lr gives another
    factor in 31 steps."""
    lr = float(np.float32(2e-3))
    dev = dict(lr=torch.tensor([lr], device=DEV))
    made = lambda: Tensors([555], eight, "f32", seed=3)   # noqa: E731
    host, others = made(), [made() for _ in range(3)]
    for step in range(1, 201):
        at = torch.tensor([step], dtype=torch.int32, device=DEV)
        host.call(step, lr=lr)
        for t, s, kw in zip(others, (step, at, at), (dev, dev, dict(lr=lr))):
            t.call(s, **kw)
            assert all(torch.equal(x, y) for x, y in zip(host.state(), t.state())), (step, kw)
