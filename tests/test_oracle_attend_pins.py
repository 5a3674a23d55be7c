"""Pins of the dense attention and rotary oracles against things other than themselves."""

import math

import numpy as np
import pytest
import torch

from oracle import sla_oracle_attend as oa
from oracle import sla_oracle_rotary as orot


def _inputs(seed, B, H, Hk, Nq, Nk, D):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(B, H, Nq, D), r(B, Hk, Nk, D), r(B, Hk, Nk, D), r(B, H, Nq, D)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq, Nk, lens", [(5, 7, [7, 3]), (7, 5, [5, 2]), (1, 6, [6, 1]), (4, 4, [0, 4])])
def test_attend_oracle_matches_autograd(causal, Nq, Nk, lens):
    B, H, Hk, D = 2, 4, 2, 8
    q, k, v, dO = _inputs(Nq + 10 * Nk, B, H, Hk, Nq, Nk, D)
    out, lse, _, _ = oa.attend(q, k, v, lens, causal)
    dq, dk, dv, *_ = oa.gradients(q, k, v, dO, lens, causal)
    a, b, c = (x.clone().requires_grad_() for x in (q, k, v))
    S = a @ b.repeat_interleave(H // Hk, 1).transpose(2, 3) / math.sqrt(D)
    keep = torch.stack([oa.visible(Nq, Nk, n, causal, "cpu") for n in lens])[:, None]
    some = keep.any(-1, keepdim=True)
    P = torch.where(some, torch.softmax(torch.where(keep, S, -1e300), -1), 0.0) * keep
    ref = P @ c.repeat_interleave(H // Hk, 1)
    ref.backward(dO)
    torch.testing.assert_close(out, ref.detach())
    torch.testing.assert_close(lse, torch.logsumexp(S.detach().masked_fill(~keep, -math.inf), -1))
    for got, x in ((dq, a), (dk, b), (dv, c)):
        torch.testing.assert_close(got, x.grad)


def test_attend_oracle_matches_central_differences():
    q, k, v, dO = _inputs(3, 1, 2, 1, 4, 6, 4)
    lens, h = [5], 1e-5
    grads = oa.gradients(q, k, v, dO, lens, True, 0.7)[:3]
    loss = lambda: float((oa.attend(q, k, v, lens, True, 0.7)[0] * dO).sum())  # noqa: E731
    for x, g in zip((q, k, v), grads):
        flat, want = x.view(-1), g.reshape(-1)
        for e in range(0, flat.numel(), 3):
            keep = float(flat[e])
            flat[e] = keep + h
            up = loss()
            flat[e] = keep - h
            down = loss()
            flat[e] = keep
            assert abs((up - down) / (2 * h) - float(want[e])) < 1e-8


def test_rows_without_keys():
    q, k, v, dO = _inputs(5, 2, 1, 1, 3, 2, 8)
    k[0], v[0] = math.nan, math.nan  # no key of the first sequence is read
    out, lse, _, _ = oa.attend(q, k, v, [0, 1], True)
    dq, dk, dv, *_ = oa.gradients(q, k, v, dO, [0, 1], True)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    assert (lse[1, 0, :2] == -math.inf).all() and lse[1, 0, 2] > -math.inf  # 3 queries, 1 key: the last sees it
    torch.testing.assert_close(out[1, 0, 2], v[1, 0, 0])
    for g in (dq, dk, dv):
        assert (g[0] == 0).all() and torch.isfinite(g).all()


def test_rotary_oracle_hand_value_and_transpose():
    x = np.array([1.0, 0.0, 0.0, 2.0]).reshape(1, 1, 1, 4)
    y = orot.rotate(x, (4,), [[1]], 100.0, 0)  # angles 1 and 0.1
    np.testing.assert_allclose(y.ravel(), [math.cos(1), math.sin(1), -2 * math.sin(0.1), 2 * math.cos(0.1)])
    rng = np.random.default_rng(0)
    x = rng.normal(size=(2, 3, 5, 12))
    pos = rng.integers(0, 99, (2, 5, 2))
    for pairing in (0, 1):
        y = orot.rotate(x, (6, 4), pos, 50.0, pairing)
        np.testing.assert_allclose(orot.rotate(y, (6, 4), pos, 50.0, pairing, -1.0), x)
        assert (y[..., 10:] == x[..., 10:]).all()


def test_rotary_scores_depend_on_differences():
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(1, 1, 1, 16)), rng.normal(size=(1, 1, 1, 16))
    s = [float((orot.rotate(q, (8, 8), [[5 + t, 9 - t]], 1e4, 1) * orot.rotate(k, (8, 8), [[2 + t, 1 - t]], 1e4, 1)).sum())
         for t in (0, 7)]
    assert abs(s[0] - s[1]) < 1e-12
    np.testing.assert_array_equal(orot.grid_positions((2, 3), (4, 0), 5), [[4, 0], [4, 1], [4, 2], [5, 0], [5, 1]])
