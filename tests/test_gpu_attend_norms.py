"""Dense attention's results by the size of their whole error.

The per-element bounds of test_gpu_attend.py add every rounding up at its worst. Here an output's whole error may be
three times what its roundings make of it in the mean square (``oracle.sla_oracle_attend.norms``): for an output of
one independent rounding that is beyond what evenly spread errors can reach (sqrt(3)), for sums of many, which are
normal, beyond 3 of their standard deviations; the mistakes planted in test_oracle_attend_mutations.py pass it tenfold."""

import pytest
import torch

from oracle import sla_oracle_attend as oa
from sparse_linear_attention_sla_b200 import binding
from tests.test_gpu_attend import SHAPES, _make

pytestmark = pytest.mark.gpu

TIMES = 3.0


def _hold(q, k, v, dO, lens=None, causal=False):
    kv = torch.tensor(lens, dtype=torch.int32, device=q.device) if lens is not None else None
    out, lse = binding.attend(q, k, v, kv, causal)
    got = (out,) + binding.attend_backward(q, k, v, out, lse, dO, kv, causal)
    refs = (oa.attend(q, k, v, lens, causal)[0],) + oa.gradients(q, k, v, dO, lens, causal)[:3]
    sizes = oa.norms(q, k, v, dO, lens, causal)
    for name, g, ref, size in zip(("out", "dq", "dk", "dv"), got, refs, sizes):
        error = float((g.double() - ref).norm())
        assert error <= TIMES * size, (name, error / size)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_whole_errors(cuda_device, shape, causal, D):
    B, H, Hk, Nq, Nk = shape
    _hold(*_make(Nq * 5 + Nk, B, H, Hk, Nq, Nk, D, cuda_device), causal=causal)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq, Nk, lens", [(200, 300, [300, 0, 1]), (64, 500, [127, 128, 129]), (300, 200, [200, 5, 130]),
                                          (1, 4000, [4000, 31, 2600]), (700, 700, [700, 383, 256])])
def test_whole_errors_with_lengths(cuda_device, Nq, Nk, lens, causal, D):
    _hold(*_make(Nq + Nk, 3, 4, 2, Nq, Nk, D, cuda_device, layout="bnhd"), lens, causal)


@pytest.mark.parametrize("q_scale", [0.1, 8.0, 60.0])
def test_whole_errors_of_flat_and_steep_rows(cuda_device, q_scale):
    q, k, v, dO = _make(3, 1, 2, 2, 200, 1100, 128, cuda_device, q_scale=q_scale)
    _hold(q, k, v, dO)
    ramp = torch.linspace(0.02, 4, 1100, device=cuda_device)
    _hold(q, (k * ramp[None, None, :, None]).to(torch.bfloat16), v, dO)
