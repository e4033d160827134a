"""The values of eps that AdamW refuses: those its reciprocal cannot take."""

import pytest
import torch

from test_training_step_host import E_UNSUP, OK, _adamw, fq, lib   # noqa: F401

REFUSED = [-1e-8, 1e-310, 1e-46, 1e-40, 2.0 ** -127, 2.0 ** 126, 1e38, 1e300, float("inf"),
           float("nan")]
TAKEN = [0.0, 2.0 ** -126, 1e-30, 1e-8, 1.0, 2.0 ** 125]


def test_the_c_abi(lib):                                                      # noqa: F811
    for eps in REFUSED:
        assert _adamw(lib, eps=eps) == E_UNSUP, eps
    for eps in TAKEN:       # (nothing to do: no device is needed)
        assert _adamw(lib, [dict(p=None, g=None, m=None, v=None, n=0)], eps=eps) == OK, eps


@pytest.mark.parametrize("eps", REFUSED)
def test_the_binding(eps):
    p, m, v = (torch.zeros(8) for _ in range(3))
    with pytest.raises(ValueError, match="eps"):
        fq.adamw([p], [torch.ones(8)], [m], [v], 1, eps=eps)
