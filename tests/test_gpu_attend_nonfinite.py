"""Dense attention on inputs that are not finite: what a NaN or an infinity enters is not finite, everything else is as
it is without it, whether a call's units are whole or cut into parts."""

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
