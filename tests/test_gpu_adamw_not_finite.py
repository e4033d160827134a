"""AdamW with moments in 8 bits where gradients are infinite, NaN or so large that their
squares overflow: those elements' moments become the code of NaN, and the others of
their group are what they are without them, bit for bit the oracle's."""

import numpy as np
import pytest

from gpu_util import host
from oracle import training_step as ots
from test_gpu_adamw import HYPER, U, Tensors

pytestmark = pytest.mark.gpu
BAD = {"inf": np.inf, "-inf": -np.inf, "nan": np.nan, "1e20": 1e20, "-1e20": -1e20, "3e38": 3e38}


def _check(t, step):
    """As Tensors.check, values that are not finite among the parameters."""
    b1, b2 = HYPER["betas"]
    for i in range(len(t.sizes)):
        with np.errstate(all="ignore"):
            m0 = ots.decode_moments(t.mq[i], t.ms[i])
            r = ots.decode_moments(t.vq[i], t.vs[i])
            m, v = ots.adamw_moments(m0, r * r, t.g[i], b1, b2)
            p, up = ots.adamw_parameters(t.p[i], m, v, step, HYPER["lr"], b1, b2,
                                         float(np.float32(HYPER["eps"])), HYPER["weight_decay"])
            root = np.sqrt(v)
        got = host(t.pd[i])
        finite = np.isfinite(p)
        assert np.array_equal(np.isfinite(got), finite)
        tol = 3 * U * np.abs(t.p[i]) + 8 * U * np.abs(up) + U * np.abs(p)
        assert np.all(np.abs(got - p)[finite] <= tol[finite])
        for x, second, qd, sd in ((m, False, t.md[i], t.msd[i]), (root, True, t.vd[i], t.vsd[i])):
            q, s = ots.encode_moments(x, step, second)
            assert np.array_equal(host(qd), q) and np.array_equal(host(sd), s)
            assert np.isfinite(host(sd)).all()
    t.p = [host(x) for x in t.pd]
    t.mq, t.ms = [host(x) for x in t.md], [host(x) for x in t.msd]
    t.vq, t.vs = [host(x) for x in t.vd], [host(x) for x in t.vsd]


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("value", list(BAD))
@pytest.mark.parametrize("at", [(3,), (130, 255), (384, 420), (0, 127, 200, 390), tuple(range(128))])
def test_neighbours_keep_their_moments(value, at, grad):
    """In the first of four steps, then with ordinary gradients: whole groups, a group's
    first and last element, the tensor's last group, a group of nothing else."""
    t = Tensors([421], True, grad, seed=7)
    plain = Tensors([421], True, grad, seed=7)
    g = t.gd[0].clone()
    t.gd[0][list(at)] = BAD[value]
    t.g[0] = host(t.gd[0].float())
    others = np.setdiff1d(np.arange(421), at)
    with np.errstate(all="ignore"):
        square = (t.g[0] * t.g[0]).astype(np.float32)
    assert not np.isfinite(square[list(at)]).any()
    for step in (9, 10, 11, 12):
        t.call(step)
        plain.call(step)
        _check(t, step)
        if step == 9:
            t.gd[0].copy_(g)
            t.g[0] = host(g.float())
        assert np.isfinite(t.p[0][others]).all()
        assert (t.vq[0][list(at)] == 0x7F).all()
        if value in ("inf", "-inf", "nan"):   # (m of the others is finite, and counts)
            assert (t.mq[0][list(at)] == 0x7F).all()
        else:
            assert np.isfinite(ots.decode_moments(t.mq[0], t.ms[0])[others]).all()
    # untouched groups are those of the call without
    clean = np.array([not set(range(128 * k, 128 * k + 128)) & set(at) for k in range(4)])
    for a, b in ((t.msd[0], plain.msd[0]), (t.vsd[0], plain.vsd[0])):
        assert np.array_equal(host(a)[clean], host(b)[clean])


def test_moments_of_32_bits_lose_the_element_alone():
    t = Tensors([300], False, "f32", seed=8)
    t.gd[0][17], t.gd[0][140] = float("inf"), float("nan")
    for step in (3, 4):
        t.call(step)
        bad = ~np.isfinite(host(t.pd[0]))
        assert np.array_equal(np.flatnonzero(bad), [17, 140])
        t.gd[0][17] = t.gd[0][140] = 0.0


def test_a_group_whose_scales_were_infinite_is_lost_as_a_whole_and_no_other():
    """State that no call writes, but that a file may hold: scales that are infinite."""
    t = Tensors([256], True, "f32", seed=9)
    t.msd[0][0] = t.vsd[0][0] = float("inf")
    t.ms, t.vs = [host(t.msd[0]).copy()], [host(t.vsd[0]).copy()]
    with np.errstate(all="ignore"):
        t.call(5)
        _check(t, 5)
    assert np.isfinite(t.p[0][128:]).all()


def test_copies_of_lost_parameters_are_nan():
    t = Tensors([200], True, "bf16", seed=10)
    t.gd[0][5] = float("nan")
    for step in (1, 2):
        t.call(step)
    copy = host(t.copies[0].float())
    assert np.isnan(copy[5]) and np.isfinite(np.delete(copy, 5)).all()
