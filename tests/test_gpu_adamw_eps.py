"""AdamW with the smallest and the largest eps that it takes."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, fq, host
from test_gpu_adamw import U
from oracle import training_step as ots

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [2.0 ** -126, 1.2e-38, 1e-37, 1e-30, 1e30, 2.0 ** 125])
def test_against_the_formula(eps):
    """Elements without a gradient ever, with one whose square underflows, with moments so
    large that their quotient by eps counts."""
    g = np.array([0, 1e-30, 1e-20, 1e-3, 1, 1e15, 0, 0] * 17, dtype=np.float32)
    m = np.array([0, 1e-38, 1e-20, 1e-3, 1, 1e37, 1e-36, 1e38] * 17, dtype=np.float32)
    v = np.zeros_like(g)
    p = np.ones_like(g)
    dev = [torch.from_numpy(t.copy()).to(DEV) for t in (p, g, m, v)]
    fq().adamw([dev[0]], [dev[1]], [dev[2]], [dev[3]], 10 ** 6, lr=1e-3, eps=eps, weight_decay=0.0)
    m2, v2 = ots.adamw_moments(m, v, g, 0.9, 0.95)
    want, up = ots.adamw_parameters(p, m2, v2, 10 ** 6, 1e-3, 0.9, 0.95, float(np.float32(eps)), 0.0)
    got = host(dev[0]).astype(np.float64)
    fits = np.abs(want) < 3e38
    tol = 3 * U * np.abs(p) + 8 * U * np.abs(up) + U * np.abs(want)
    assert np.all(np.abs(got - want)[fits] <= tol[fits])
    assert not np.isfinite(got[~fits]).any() and np.all(got[::8] == 1)


@pytest.mark.parametrize("eps", [1e-46, 1e-40, 2.0 ** 126])
def test_refused_before_anything_is_written(eps):
    for kw in (dict(), dict(stream=torch.cuda.current_stream())):
        p, m, v = (torch.zeros(8, device=DEV) for _ in range(3))
        with pytest.raises(ValueError, match="eps"):
            fq().adamw([p], [torch.ones(8, device=DEV)], [m], [v], 1, eps=eps, **kw)
        assert not (p.any() or m.any() or v.any())
