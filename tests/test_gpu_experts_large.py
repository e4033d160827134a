"""Tokens by expert and the gated backward pass by expert where operands and results pass
2^32 bytes: the last rows, compared with a call of their own."""

import torch
import pytest

from gpu_util import DEV, fq

pytestmark = pytest.mark.gpu
M, TAIL = 300_007, 300


def _offsets(rows_before):
    at = [0, rows_before, rows_before + 50, rows_before + 50, rows_before + TAIL - 3]
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _rows(width):
    x = torch.zeros((M, width), dtype=torch.bfloat16, device=DEV)
    x[-TAIL:] = torch.randn((TAIL, width), device=DEV).to(torch.bfloat16)
    return x


def _check_columns(whole, tail):
    """Codes and scales of both calls' groups; what lies before and behind is zeros."""
    (q, s), (tq, ts) = whole, tail
    first = (M - TAIL + 127) // 128
    n = min(ts.shape[0], s.shape[0] - first)
    assert torch.equal(s[first:first + n], ts[:n])
    assert torch.equal(q[:, 128 * first:128 * (first + n)], tq[:, :128 * n])
    assert not s[:first].any() and not s[first + n:].any() and not ts[n:].any()
    assert not q[-1, :128 * first].any() and not q[0, :128 * first].any()


def test_tokens_by_expert():
    K = 16384
    x = _rows(K)
    whole = fq().grouped_quantize_act_t(x, _offsets(M - TAIL))
    assert whole[0].numel() > 1 << 32
    _check_columns(whole, fq().grouped_quantize_act_t(x[-TAIL:], _offsets(0)))


def test_gated_backward_by_expert():
    F = 8192
    dh, gu = _rows(F), _rows(2 * F)
    q, s, qt, st = fq().grouped_gated_backward(dh, gu, _offsets(M - TAIL))
    assert q.numel() > 1 << 32 and qt.numel() > 1 << 32
    tq, ts, tqt, tst = fq().grouped_gated_backward(dh[-TAIL:], gu[-TAIL:], _offsets(0))
    live = TAIL - 3
    assert torch.equal(q[-TAIL:][:live], tq[:live]) and torch.equal(s[:, -TAIL:][:, :live], ts[:, :live])
    assert not q[:128].any() and not s[:, :M - TAIL].any()
    _check_columns((qt, st), (tqt, tst))
