"""Dense attention on inputs that are not finite, and on finite scores of any size: what a NaN or an infinity enters is
not finite, everything else is as it is without it, whether a call's units are whole or cut into parts."""

import math

import pytest
import torch

from sparse_linear_attention_sla_b200 import binding

pytestmark = pytest.mark.gpu

B, H, HK, D = 2, 4, 2, 128

# Nq, Nk, lens: units of one tile and of two, whole (few steps) and cut into parts (many steps, or lengths).
CALLS = [(64, 128, None), (300, 300, None), (1, 4000, None), (1, 4000, [4000, 2600]), (64, 2000, None),
         (300, 3000, None), (300, 3000, [3000, 1111]), (130, 260, [260, 131])]


def _make(seed, Nq, Nk, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    one = lambda h, n: torch.randn(B, h, n, D, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    return one(H, Nq), one(HK, Nk), one(HK, Nk), one(H, Nq)


def _lens(lens, dev):
    return torch.tensor(lens, dtype=torch.int32, device=dev) if lens else None


def _same(got, want, but):
    """got is want except at the rows `but`."""
    return torch.equal(got.masked_fill(but, 0), want.masked_fill(but, 0))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq, Nk, lens", CALLS)
def test_a_query_row_of_nan(cuda_device, Nq, Nk, lens, causal):
    q, k, v, dO = _make(Nq + Nk, Nq, Nk, cuda_device)
    kv = _lens(lens, cuda_device)
    want, wlse = binding.attend(q, k, v, kv, causal)
    clean = binding.attend_backward(q, k, v, want, wlse, dO, kv, causal)
    i = Nq - 1
    q[1, 2, i] = math.nan
    bad = torch.zeros(B, H, Nq, dtype=torch.bool, device=cuda_device)
    bad[1, 2, i] = True
    out, lse = binding.attend(q, k, v, kv, causal)
    assert out[1, 2, i].isnan().all() and lse[1, 2, i].isnan()
    assert _same(out, want, bad[..., None]) and _same(lse, wlse, bad)
    dq, dk, dv = binding.attend_backward(q, k, v, out, lse, dO, kv, causal)
    n = lens[1] if lens else Nk
    assert dq[1, 2, i].isnan().all() and dk[1, 1, :n].isnan().all() and dv[1, 1, :n].isnan().all()  # the last row sees every key
    for got, ref in ((dq, clean[0]), (dk, clean[1]), (dv, clean[2])):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1, 0], ref[1, 0])  # other sequences and heads


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq, Nk, lens", CALLS)
def test_one_key_of_nan(cuda_device, Nq, Nk, lens, causal):
    q, k, v, dO = _make(Nq + 2 * Nk, Nq, Nk, cuda_device)
    kv = _lens(lens, cuda_device)
    want, wlse = binding.attend(q, k, v, kv, causal)
    n = lens[1] if lens else Nk
    j = n - 1 - min(Nq, n) // 2
    k[1, 1, j] = math.nan
    i = torch.arange(Nq, device=cuda_device)
    bad = torch.zeros(B, H, Nq, dtype=torch.bool, device=cuda_device)
    bad[1, 2:] = (j <= i + n - Nq) if causal else True
    assert bad.any()
    out, lse = binding.attend(q, k, v, kv, causal)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert _same(out, want, bad[..., None]) and _same(lse, wlse, bad)
    dq, dk, dv = binding.attend_backward(q, k, v, out, lse, dO, kv, causal)
    assert dq[bad].isnan().all() and dk[1, 1, :n].isnan().all() and dv[1, 1, :n].isnan().all()
    assert torch.isfinite(dq[0]).all() and torch.isfinite(dk[1, 0]).all()


@pytest.mark.parametrize("Nq, Nk, lens", CALLS)
def test_infinite_scores(cuda_device, Nq, Nk, lens):
    """A key whose first channel is infinite: a score of +inf leaves no number, one of -inf has no weight."""
    q, k, v, _ = _make(3 * Nq + Nk, Nq, Nk, cuda_device)
    kv = _lens(lens, cuda_device)
    j = (lens[1] if lens else Nk) // 2
    hidden = k.clone()
    hidden[1, 1, j, 0] = -3e4  # q[.., 0] > 0.1: a weight of 2^-100 at most, no number of bf16 beside 1
    k[1, 1, j, 0] = math.inf
    q[..., 0] = q[..., 0].abs().clamp(min=0.5)
    out, lse = binding.attend(q, k, v, kv)
    assert out[1, 2:].isnan().all() and not torch.isfinite(lse[1, 2:]).any()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :2]).all() and torch.isfinite(lse[1, :2]).all()
    k[1, 1, j, 0] = -math.inf
    out, lse = binding.attend(q, k, v, kv)
    want, wlse = binding.attend(q, hidden, v, kv)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


# Magnitudes of the scores: below and above where half a step of the largest, in base 2, is 128.
SIZES = (2.0 ** 24, 2.0 ** 29, 2.0 ** 31, 2.0 ** 33, 2.0 ** 36, 1e20, 1e37)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("Nq, Nk", [(64, 128), (300, 300), (1, 4000), (300, 1500)])
def test_finite_scores_of_any_size(cuda_device, Nq, Nk, sign):
    """Scores c k_j of distinct k_j, exact in fp32: the row is one-hot, out the value of the largest score and lse that
    score, off by the rounding of the score, of the scale and of two products (2^-22 of it), wherever it lies and
    whatever the rows beside it hold."""
    q, k, v, _ = _make(7 * Nq + Nk, Nq, Nk, cuda_device)
    g = torch.Generator().manual_seed(Nq + Nk)
    rows = min(Nq, len(SIZES) * 3)
    for b in range(B):
        for h in range(HK):  # distinct bf16 numbers from -1 up and from 1 down, in some order
            n = torch.randperm(Nk, generator=g)
            size = (0x3f80 - n // 2).to(torch.int16).view(torch.bfloat16)
            k[b, h, :, 0] = torch.where(n % 2 == 0, size, -size).to(cuda_device)
    q[..., 0] = 0
    want, wlse = binding.attend(q, k, v)
    for r in range(rows):
        q[:, :, r] = 0
        q[:, :, r, 0] = sign * SIZES[(r + Nk) % len(SIZES)]
    out, lse = binding.attend(q, k, v)
    assert torch.equal(out[:, :, rows:], want[:, :, rows:]) and torch.equal(lse[:, :, rows:], wlse[:, :, rows:])
    first = k[..., 0].double()
    at = (first * sign).argmax(-1)  # [B, HK]
    for b in range(B):
        for h in range(H):
            best = at[b, h // (H // HK)]
            assert torch.equal(out[b, h, :rows], v[b, h // (H // HK), best].expand(rows, D)), (b, h)
            ref = q[b, h, :rows, 0].double() * first[b, h // (H // HK), best] / D ** 0.5
            assert ((lse[b, h, :rows].double() - ref).abs() <= 2.0 ** -22 * ref.abs()).all()


def test_references_that_leave_and_enter_the_largest_sizes(cuda_device):
    """The first keys' scores are huge and negative, then ordinary; ordinary, then huge; equal huge ones share a row."""
    q, k, v, _ = _make(77, 200, 1000, cuda_device)
    q[..., 0], k[..., 0] = 1e18, 0
    low = k.clone()
    low[:, :, :300, 0] = -1e18
    out, lse = binding.attend(q, low, v)
    want, wlse = binding.attend(q, k[:, :, 300:], v[:, :, 300:])
    tol = 2.0 ** -7 * v.float().abs().max()  # of each call: a rounding of P and one of out, by 2^-8 of |v| at most
    assert ((out.float() - want.float()).abs() <= 2 * tol).all()
    assert ((lse - wlse).abs() <= 2.0 ** -20 * (1 + wlse.abs())).all()
    k[:, :, 500, 0] = k[:, :, 900, 0] = 1e18
    k[:, :, [500, 900], 1:] = 0
    out, lse = binding.attend(q, k, v)
    mean = (v[:, :, 500].float() + v[:, :, 900].float()).repeat_interleave(H // HK, 1)[:, :, None] / 2
    assert ((out.float() - mean).abs() <= 2.0 ** -8 * mean.abs()).all()
