"""The example's captured training of experts against the same steps called one by one."""

import pytest
import torch

from test_gpu_training_step import BF16, ROUTES, _offsets, _rows, _same, _state, example   # noqa: F401

pytestmark = pytest.mark.gpu


def test_training_is_the_eager_steps(example):                                     # noqa: F811
    """Six steps of train_experts, five of them replays, leave the state and give the two
    losses of six eager steps, bit for bit."""
    hidden, x, off, lr, steps = 256, _rows(5, 256, 256), _offsets(ROUTES[0]), 1e-3, 6
    target, layer, twin = (example.ExpertLayer(hidden, 128, 4, s) for s in (20, 21, 21))
    start = [t.clone() for t in _state(layer)]
    first, last = example.train_experts(layer, target, x, off, steps, lr)
    want, losses = target.forward(x, off).float(), []
    for _ in range(steps):
        e = twin.forward(x, off).float() - want
        losses.append(float(e.square().mean()))
        _, dw, dnorm = twin.backward((e * (2.0 / hidden)).to(BF16))
        twin.update(dw, dnorm, lr)
    torch.cuda.synchronize()
    assert (first, last) == (losses[0], losses[-1])
    assert _same(_state(layer), _state(twin)) and not _same(_state(layer), start)
