"""What the dense attention's and the rotary positions' oracles are held to beside their own pins: torch's attention,
rotation matrices, and mistakes planted in an implementation that rounds as the kernels do, each of which has to pass
the tolerances that the GPU tests use."""

import math

import numpy as np
import pytest
import torch

from oracle import sla_oracle_attend as oa
from oracle import sla_oracle_rotary as orot

TIMES = 3.0  # what the whole error may be of its expected size, as in the GPU tests


def _inputs(seed, B, H, Hk, Nq, Nk, D, q_scale=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, n, s=1.0: (torch.randn(B, h, n, D, generator=g) * s).to(torch.bfloat16)  # noqa: E731
    return r(H, Nq, q_scale), r(Hk, Nk), r(Hk, Nk), r(H, Nq)


def _b(x):
    return x.to(torch.bfloat16).float()


def rounded(q, k, v, dO, lens=None, causal=False, scale=None, mistake=None):
    """out, lse and the gradients as the kernels form them: P, T and the results rounded to bf16, the rest fp32, delta from
    the rounded out; with one mistake."""
    B, H, Nq, D = q.shape
    Hk, Nk = k.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    out, dq = torch.zeros(B, H, Nq, D), torch.zeros(B, H, Nq, D)
    dk, dv = torch.zeros(B, Hk, Nk, D), torch.zeros(B, Hk, Nk, D)
    lse = torch.full((B, H, Nq), -math.inf)
    for b in range(B):
        n = Nk if lens is None else lens[b]
        for h in range(H):
            kh = h // (H // Hk)
            Q, K, V, G = q[b, h].float(), k[b, kh, :n].float(), v[b, kh, :n].float(), dO[b, h].float()
            keep = oa.visible(Nq, n, n, causal, "cpu")
            if mistake == "mask of one key more" and causal:
                keep = torch.cat([keep[1:], keep[-1:]])
            S = (Q @ K.T * scale).masked_fill(~keep, -math.inf)
            if mistake == "a key tile skipped":
                S[:, 128:256] = -math.inf
            m = S.amax(1, keepdim=True)
            p = torch.where(m == -math.inf, 0.0, torch.exp(S - m))
            l = p.sum(1, keepdim=True)
            live = l > 0
            some = torch.where(live, l, 1.0)
            out[b, h] = _b(_b(p) @ V / some)
            lse[b, h] = torch.where(live, m + l.log(), -math.inf)[:, 0]
            P = p / some
            delta = (G * out[b, h]).sum(1, keepdim=True)
            if mistake == "delta dropped":
                delta = torch.zeros_like(delta)
            if mistake == "delta of the wrong sign":
                delta = -delta
            T = _b(P * (G @ V.T - delta))
            P = _b(P)
            s = {"scale missing": 1.0, "scale off by a tenth": 1.1 * scale}.get(mistake, scale)
            dq[b, h] = _b(s * T @ K)
            if mistake == "a query head left out of dk" and h == 1:
                continue
            rows = slice(128, None) if mistake == "a query tile skipped" else slice(None)
            half = slice(None, n // 2 // 128 * 128) if mistake == "a part not joined" else slice(None)
            dk[b, kh, :n][half] += s * T[rows].T[half] @ Q[rows]
            dv[b, kh, :n][half] += P[rows].T[half] @ G[rows]
    return out, lse, dq, _b(dk), _b(dv)


PROBLEMS = [
    # B, H, Hk, Nq, Nk, lens, causal
    (1, 4, 2, 300, 500, None, False),
    (2, 2, 1, 260, 400, [400, 300], True),
]


def _errors(p, mistake=None, **kw):
    B, H, Hk, Nq, Nk, lens, causal = p
    q, k, v, dO = _inputs(Nq + Nk, B, H, Hk, Nq, Nk, 64, **kw)
    got = rounded(q, k, v, dO, lens, causal, mistake=mistake)
    ref, rlse, bound, lbound = oa.attend(q, k, v, lens, causal)
    grads = oa.gradients(q, k, v, dO, lens, causal)
    size = oa.norms(q, k, v, dO, lens, causal)
    refs, bounds = (ref,) + grads[:3], (bound,) + grads[3:]
    got = (got[0],) + got[2:]
    return {name: (float((g.double() - r).norm()) / s, bool(((g.double() - r).abs() <= b).all()))
            for name, g, r, b, s in zip(("out", "dq", "dk", "dv"), got, refs, bounds, size)}


@pytest.mark.parametrize("q_scale", [1.5, 20.0])
@pytest.mark.parametrize("p", PROBLEMS)
def test_an_implementation_that_rounds_so_is_within(p, q_scale):
    """And not far inside: its errors are at least a quarter of the expected ones."""
    for name, (times, inside) in _errors(p, q_scale=q_scale).items():
        assert inside and 0.25 <= times <= TIMES / 2, (name, times)


@pytest.mark.parametrize("mistake, seen", [
    ("a key tile skipped", ("out", "dq", "dk", "dv")), ("delta dropped", ("dq", "dk")),
    ("delta of the wrong sign", ("dq", "dk")), ("scale missing", ("dq", "dk")), ("scale off by a tenth", ("dq", "dk")),
    ("a query head left out of dk", ("dk", "dv")), ("a query tile skipped", ("dk", "dv")),
    ("a part not joined", ("dk", "dv")), ("mask of one key more", ("out", "dq", "dk", "dv")),
])
@pytest.mark.parametrize("p", PROBLEMS)
def test_planted_mistakes_pass_the_norms(p, mistake, seen):
    if mistake == "mask of one key more":
        p = p[:6] + (True,)
    errors = _errors(p, mistake)
    for name in seen:
        assert errors[name][0] > TIMES, (name, errors[name])


@pytest.mark.parametrize("mistake, seen", [
    ("a key tile skipped", ("out", "dq", "dk", "dv")), ("scale missing", ("dq", "dk")),
    ("a query head left out of dk", ("dk", "dv")), ("a query tile skipped", ("dk", "dv")), ("a part not joined", ("dk", "dv")),
])
@pytest.mark.parametrize("p", PROBLEMS)
def test_planted_mistakes_pass_the_bounds(p, mistake, seen):
    errors = _errors(p, mistake)
    for name in seen:
        assert not errors[name][1], name


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq, Nk", [(7, 7), (5, 12)])
def test_attend_oracle_is_torchs_attention(Nq, Nk, causal):
    """scaled_dot_product_attention with the mask spelt out, keys shared by repetition."""
    q, k, v, _ = (x.double() for x in _inputs(3, 2, 4, 2, Nq, Nk, 16))
    lens = [Nk, Nk - 1 if causal else 3]
    mask = torch.stack([torch.arange(Nk) < n for n in lens])[:, None, None]
    if causal:
        shift = torch.tensor(lens)[:, None, None, None] - Nq
        mask = mask & (torch.arange(Nk) <= torch.arange(Nq)[:, None] + shift)
    want = torch.nn.functional.scaled_dot_product_attention(q, k.repeat_interleave(2, 1), v.repeat_interleave(2, 1),
                                                            attn_mask=mask.expand(2, 4, Nq, Nk), scale=0.3)
    got = oa.attend(q, k, v, lens, causal, 0.3)[0]
    rows = mask.expand(2, 4, Nq, Nk).any(-1)
    torch.testing.assert_close(got[rows], want[rows])


def test_rotary_oracle_is_a_rotation_matrix():
    """Every pair by its 2 x 2 matrix, written out; a planted wrong frequency, sign or pairing is seen."""
    rng = np.random.default_rng(2)
    axes, base = (6, 4), 30.0
    x = rng.normal(size=(2, 2, 4, 12))
    pos = rng.integers(-9, 99, (4, 2))
    for pairing in (0, 1):
        want = x.copy()
        for n in range(4):
            first = 0
            for a, d in enumerate(axes):
                for i in range(d // 2):
                    phi = pos[n, a] / base ** (2 * i / d)
                    m = np.array([[np.cos(phi), -np.sin(phi)], [np.sin(phi), np.cos(phi)]])
                    c = [first + 2 * i, first + 2 * i + 1] if pairing == 0 else [first + i, first + i + d // 2]
                    want[:, :, n, c] = x[:, :, n, c] @ m.T
                first += d
        np.testing.assert_allclose(orot.rotate(x, axes, pos, base, pairing), want, atol=1e-12)
        for wrong in (orot.rotate(x, axes, pos, base * 1.01, pairing), orot.rotate(x, axes, pos, base, pairing, -1.0),
                      orot.rotate(x, axes, pos, base, 1 - pairing), orot.rotate(x, axes, pos + 1, base, pairing)):
            assert np.abs(wrong - want).max() > 1e-2
