"""The positions and the attentions as a model's layers run them: rotation, attention, the attention's gradients
and the rotation's transpose, and the sparse attention's own paths with rotary_by."""

import numpy as np
import pytest
import torch

from oracle import sla_oracle_attend as oa
from oracle import sla_oracle_rotary as orot
from sparse_linear_attention_sla_b200 import binding
from sparse_linear_attention_sla_b200.workloads import random_inputs

pytestmark = pytest.mark.gpu

AXES, GRID = (44, 42, 42), (3, 8, 11)


def _projections(dev, B, N, heads, D, seed):
    """What projections leave: [B, N, H, D] tensors, seen as [B, H, N, D]."""
    g = torch.Generator(device=dev).manual_seed(seed)
    return [torch.randn(B, N, h, D, generator=g, device=dev).to(torch.bfloat16).transpose(1, 2) for h in heads]


def test_rotary_attend_and_back(cuda_device):
    """Every step's result is the next step's input; each is held to the oracle of that step on the inputs it had."""
    B, N, H, Hk, D = 2, 264, 4, 2, 128
    q, k, v, dO = _projections(cuda_device, B, N, (H, Hk, Hk, H), D, 1)
    spec = binding.rotary_spec(AXES, grid=GRID)
    lens = torch.tensor([264, 129], dtype=torch.int32, device=cuda_device)
    qr, kr = binding.rotary(q, k, spec)
    out, lse = binding.attend(qr, kr, v, lens)
    dqr, dkr, dv = binding.attend_backward(qr, kr, v, out, lse, dO, lens)
    dq, dk = binding.rotary_backward(dqr, dkr, spec)
    ref, _, bound, _ = oa.attend(qr, kr, v, lens.tolist())
    assert ((out.double() - ref).abs() <= bound).all()
    refs = oa.gradients(qr, kr, v, dO, lens.tolist())
    for got, r, b in zip((dqr, dkr, dv), refs[:3], refs[3:]):
        assert ((got.double() - r).abs() <= b).all()
    pos = orot.grid_positions(GRID, (0, 0, 0), N)
    for got, x in ((qr, q), (kr, k)):
        want = orot.rotate(x.double().cpu().numpy(), AXES, pos, 1e4, 0)
        size = np.abs(want).max()
        assert np.abs(got.double().cpu().numpy() - want).max() <= 2.0 ** -8 * size + 2.0 ** -20 * size
    for got, x in ((dq, dqr), (dk, dkr)):
        want = orot.rotate(x.double().cpu().numpy(), AXES, pos, 1e4, 0, -1.0)
        size = np.abs(want).max()
        assert np.abs(got.double().cpu().numpy() - want).max() <= 2.0 ** -8 * size + 2.0 ** -20 * size


@pytest.mark.parametrize("pairing", [0, 1])
def test_sparse_forward_and_backward_by_rotary(cuda_device, pairing):
    B, H, N, D = 1, 2, 264, 128
    q, k, v, dO = _projections(cuda_device, B, N, (H,) * 4, D, 2)
    v, dO = v.contiguous(), dO.contiguous()
    alpha = random_inputs(B, H, N, D, seed=3, device=cuda_device)[3]
    spec = binding.rotary_spec(AXES, grid=GRID, pairing=pairing)
    qr, kr = binding.rotary(q, k, spec)
    args = dict(block_q=128, block_kv=64, kh=0.3, kl=0.2)
    assert torch.equal(binding.forward(q, k, v, alpha, **args, rotary_by=spec), binding.forward(qr, kr, v, alpha, **args))
    assert torch.equal(binding.forward_fp8(q, k, v, alpha, **args, rotary_by=spec),
                       binding.forward_fp8(qr, kr, v, alpha, **args))
    assert torch.equal(binding.forward_pisa(q, k, v, **args, rotary_by=spec), binding.forward_pisa(qr, kr, v, **args))
    assert torch.equal(binding.forward_variant(q, k, v, alpha, 128, 64, 0.3, 0.2, feature_map=1, rotary_by=spec),
                       binding.forward_variant(qr, kr, v, alpha, 128, 64, 0.3, 0.2, feature_map=1))
    got = binding.backward(q, k, v, alpha, dO, **args, rotary_by=spec)
    binding.check(got[4])
    want = binding.backward(qr, kr, v, alpha, dO, **args)
    for a, b in zip(got[:2], binding.rotary_backward(want[0], want[1], spec)):
        assert a.dtype == torch.float32 and torch.equal(a, b)
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
    low = binding.rotary_backward(want[0], want[1], spec, dtype=torch.bfloat16)
    assert torch.equal(low[0], got[0].to(torch.bfloat16)) and torch.equal(low[1], got[1].to(torch.bfloat16))


def test_dense_sparse_attention_and_attend_agree(cuda_device):
    """With every block critical and alpha = 1 the sparse attention is the dense one: both are within the dense oracle's
    bound of it (the sparse kernel rounds P and its output once each, as attend does)."""
    q, k, v, _ = random_inputs(1, 2, 500, 128, seed=4, device=cuda_device)
    alpha = torch.ones(2, 128, device=cuda_device)
    dense, _ = binding.attend(q, k, v)
    sparse = binding.forward(q, k, v, alpha, 128, 64, 1.0, 0.0)
    ref, _, bound, _ = oa.attend(q, k, v)
    assert ((dense.double() - ref).abs() <= bound).all()
    assert ((sparse.double() - ref).abs() <= bound + 2.0 ** -24 * v.double().abs().max()).all()


def test_offsets_past_32_bits(cuda_device):
    """Rows that lie 24 MB apart: the last ones past 4 GB."""
    dev, N, step = cuda_device, 200, 12 * 2 ** 20
    room = torch.empty(N * step, dtype=torch.bfloat16, device=dev)

    def apart(x, at):
        y = room.as_strided((1, x.shape[1], N, 128), (N * step, 128, step, 1), at)
        y.copy_(x)
        return y

    q, k, v, dO = (x.contiguous() for x in _projections(dev, 1, N, (2, 2, 2, 2), 128, 5))
    Q, K, V, G = (apart(x, 1024 * i) for i, x in enumerate((q, k, v, dO)))
    out, lse = binding.attend(Q, K, V, causal=True)
    want = binding.attend(q, k, v, causal=True)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    O = room.as_strided((1, 2, N, 128), (N * step, 128, step, 1), 8192)
    binding.attend(Q, K, V, causal=True, out=O)
    assert torch.equal(O, want[0])
    for a, b in zip(binding.attend_backward(Q, K, V, O, lse, G, causal=True),
                    binding.attend_backward(q, k, v, *want, dO, causal=True)):
        assert torch.equal(a, b)
    spec = binding.rotary_spec((128,), grid=(N,), pairing=1)
    for a, b in zip(binding.rotary(Q, K, spec), binding.rotary(q, k, spec)):
        assert torch.equal(a, b)
    binding.rotary(Q, K, spec, out=(Q, K))
    assert torch.equal(Q, binding.rotary(q, k, spec)[0])
