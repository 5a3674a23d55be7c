"""GPU parity of the rotary positions against the fp64 oracle.

A value is formed in fp32 from an angle that is reduced in 64 bits: cos and sin are off by at most
2^-22 (their argument, at most pi, is rounded to fp32 by 2^-23, and sincosf by 2 steps), the two
products and their sum by 2^-24 each, so |error| <= 2^-21 (|x1| + |x2|), plus half a bf16 step
(2^-8 of the value) where the result is bf16.
"""

import math

import numpy as np
import pytest
import torch

from oracle import sla_oracle_rotary as orot
from sparse_linear_attention_sla_b200 import binding

pytestmark = pytest.mark.gpu


def _within(got, x, axes, positions, base, pairing, sign=1.0):
    x64 = x.double().cpu().numpy()
    ref = orot.rotate(x64, axes, positions, base, pairing, sign)
    size = orot.rotate(np.abs(x64), axes, np.zeros(np.asarray(positions).shape), base, pairing)
    other = size.copy()
    first = 0
    for d in axes:
        i = np.arange(d // 2)
        c1, c2 = (first + 2 * i, first + 2 * i + 1) if pairing == 0 else (first + i, first + i + d // 2)
        other[..., c1], other[..., c2] = size[..., c2], size[..., c1]
        first += d
    bound = 2.0 ** -21 * (size + other) + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0.0)
    d = np.abs(got.double().cpu().numpy() - ref)
    assert np.isfinite(d).all()
    assert (d <= bound).all(), float((d - bound).max())


def _make(seed, B, H, N, D, dtype, dev, layout="bnhd"):
    g = torch.Generator(device=dev).manual_seed(seed)
    if layout == "bnhd":
        return torch.randn(B, N, H, D, generator=g, device=dev).to(dtype).transpose(1, 2)
    return torch.randn(B, H, N, D, generator=g, device=dev).to(dtype)


@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("D, axes, grid, N", [
    (128, (44, 42, 42), (3, 5, 7), 105), (128, (44, 42, 42), (3, 5, 7), 110), (128, (128,), (40,), 33),
    (64, (24, 20, 20), (2, 3, 4), 24), (64, (16, 8), (5, 3), 17), (64, (32, 32), (1, 1), 3),
    (128, (32, 32, 32, 32), (2, 2, 2, 3), 24), (64, (2,), (70,), 67), (64, (64,), (1,), 1),
])
def test_grid(cuda_device, D, axes, grid, N, pairing):
    start = tuple(range(5, 5 + len(axes)))
    q, k = _make(N, 2, 5, N, D, torch.bfloat16, cuda_device), _make(N + 1, 2, 2, N, D, torch.bfloat16, cuda_device)
    spec = binding.rotary_spec(axes, grid=grid, start=start, base=1e4, pairing=pairing)
    pos = orot.grid_positions(grid, start, N)
    for got, x in zip(binding.rotary(q, k, spec), (q, k)):
        assert got.is_contiguous()
        _within(got, x, axes, pos, 1e4, pairing)
        assert torch.equal(got[:, :, len(pos):], x[:, :, len(pos):])      # behind the grid
        assert torch.equal(got[..., sum(axes):], x[..., sum(axes):])      # channels of no axis


@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("dtype, out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                        (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("shared", [False, True])
def test_positions_and_backward(cuda_device, dtype, out, shared, pairing):
    B, N, D, axes = 3, 45, 128, (44, 42, 42)
    g = torch.Generator(device=cuda_device).manual_seed(4)
    pos = torch.randint(-50, 2 ** 31 - 1, (N, 3) if shared else (B, N, 3), generator=g, device=cuda_device,
                        dtype=torch.int32)
    q, k = _make(1, B, 3, N, D, dtype, cuda_device), _make(2, B, 1, N, D, dtype, cuda_device, "bhnd")
    spec = binding.rotary_spec(axes, positions=pos, base=1e6, pairing=pairing)
    # an fp64 angle of up to 2^31 is itself off by 2^-23: keep the positions where it is not
    small = binding.rotary_spec(axes, positions=pos % 1000003, base=1e6, pairing=pairing)
    for got, x in zip(binding.rotary_backward(q, k, small, dtype=out), (q, k)):
        assert got.dtype == out
        _within(got, x, axes, (pos % 1000003).cpu().numpy(), 1e6, pairing, -1.0)
    if dtype == out:
        for got, x in zip(binding.rotary(q, k, small), (q, k)):
            _within(got, x, axes, (pos % 1000003).cpu().numpy(), 1e6, pairing)
        for got, x in zip(binding.rotary(q, k, spec), (q, k)):  # any int32 position: lengths stay
            assert torch.isfinite(got).all()
            a, b = got.double().square().sum(-1), x.double().square().sum(-1)
            assert ((a - b).abs() <= 2.0 ** (-6 if out == torch.bfloat16 else -19) * b).all()


@pytest.mark.parametrize("pairing", [0, 1])
def test_in_place_and_single(cuda_device, pairing):
    q, k = _make(7, 1, 4, 50, 64, torch.bfloat16, cuda_device), _make(8, 1, 2, 50, 64, torch.bfloat16, cuda_device)
    spec = binding.rotary_spec((24, 20, 20), grid=(2, 5, 5), pairing=pairing)
    want = binding.rotary(q, k, spec)
    assert torch.equal(binding.rotary(q, None, spec)[0], want[0])
    assert torch.equal(binding.rotary(None, k, spec)[1], want[1])
    packed = torch.cat([q.transpose(1, 2), k.transpose(1, 2)], dim=2).contiguous()
    a, b = packed[:, :, :4].transpose(1, 2), packed[:, :, 4:].transpose(1, 2)
    got = binding.rotary(a, b, spec, out=(a, b))
    assert got[0].data_ptr() == a.data_ptr()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_neighbours_of_copied_channels(cuda_device):
    """NaN and infinities in channels that turn leave those that do not as they were."""
    x = _make(9, 1, 2, 9, 64, torch.bfloat16, cuda_device)
    x[..., 16:20] = math.inf
    x[0, 0, 3, :16] = math.nan
    for pairing in (0, 1):
        spec = binding.rotary_spec((16,), grid=(5,), pairing=pairing)
        y, _ = binding.rotary(x, None, spec)
        assert torch.equal(y[..., 16:], x[..., 16:])
        assert torch.equal(y[:, :, 5:].nan_to_num(5.0), x[:, :, 5:].nan_to_num(5.0))
        assert torch.isfinite(y[:, 1, :, :16]).all()


def test_captured_and_replayed(cuda_device):
    q, k = _make(3, 2, 3, 40, 128, torch.bfloat16, cuda_device), _make(4, 2, 3, 40, 128, torch.bfloat16, cuda_device)
    pos = torch.arange(40, dtype=torch.int32, device=cuda_device)[:, None].contiguous()
    spec = binding.rotary_spec((128,), positions=pos, pairing=1)
    binding.rotary(q, k, spec)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = binding.rotary(q, k, spec)
    pos.mul_(3)
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    want = binding.rotary(q, k, spec)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_in_place_within_one_projection(cuda_device):
    """q and k as slices of one [B, N, 3, H, D] buffer, turned where they lie; v between them stays as it was."""
    buf = torch.randn(2, 50, 3, 4, 64, device=cuda_device, generator=torch.Generator(cuda_device).manual_seed(8))
    buf = buf.to(torch.bfloat16)
    q, v, k = (buf[:, :, i].transpose(1, 2) for i in range(3))
    spec = binding.rotary_spec((32, 32), grid=(5, 10))
    want, kept = binding.rotary(q, k, spec), v.clone()
    binding.rotary(q, k, spec, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)
    with pytest.raises(ValueError):
        binding.rotary(q, k, spec, out=(q, buf[:, :, 1:].flatten(2, 3)[:, :, 2:6].transpose(1, 2)))  # half of v, half of k


def test_refusals(cuda_device):
    x = _make(1, 1, 2, 10, 64, torch.bfloat16, cuda_device)
    ok = binding.rotary_spec((64,), grid=(10,))
    pos = torch.zeros(10, 1, dtype=torch.int32, device=cuda_device)
    bad = [
        lambda: binding.rotary_spec((64,)),
        lambda: binding.rotary_spec((64,), grid=(10,), positions=pos),
        lambda: binding.rotary_spec((32, 32), grid=(10,)),
        lambda: binding.rotary_spec((64,), positions=pos.long()),
        lambda: binding.rotary_spec((8,) * 5, grid=(1,) * 5),
        lambda: binding.rotary(x, None, binding.rotary_spec((63,), grid=(10,))),
        lambda: binding.rotary(x, None, binding.rotary_spec((64, 2), grid=(5, 2))),
        lambda: binding.rotary(x, None, binding.rotary_spec((64,), grid=(0,))),
        lambda: binding.rotary(x, None, binding.rotary_spec((64,), grid=(10,), base=0.0)),
        lambda: binding.rotary(x, None, binding.rotary_spec((64,), grid=(10,), pairing=2)),
        lambda: binding.rotary(x, None, binding.rotary_spec((64,), positions=pos[:9].contiguous())),
        lambda: binding.rotary(None, None, ok),
        lambda: binding.rotary(x.half(), None, ok),
        lambda: binding.rotary(x[..., :32], None, ok),
        lambda: binding.rotary(x, x[:, :, :9], ok),
        lambda: binding.rotary_backward(x, None, ok, dtype=torch.float32),
        lambda: binding.rotary(x[:, :, 1:], None, binding.rotary_spec((64,), grid=(9,)), out=(x[:, :, :9], None)),
        lambda: binding.rotary(x.cpu(), None, ok),
        lambda: binding.rotary(x, x.clone(), ok, out=(x, x)),
        lambda: binding.rotary_spec((64,), grid=(2 ** 32 + 10,)),
        lambda: binding.rotary_spec((64,), grid=(10,), start=(2 ** 31,)),
    ]
    for f in bad:
        with pytest.raises((ValueError, binding.SlaError)):
            f()
    assert torch.isfinite(binding.rotary(x, None, ok)[0]).all()
