"""Dense attention's gradients against differences of its own forward, along directions in which a mistake shows."""

import math

import pytest
import torch

from oracle import sla_oracle_attend as oa
from sparse_linear_attention_sla_b200 import binding
from tests.test_gpu_attend import _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 64])
def test_differences_along_the_gradients(cuda_device, D):
    """Central differences of the kernel's own forward, over steps of length 2 along a gradient and along what a gradient
    without delta would be off by.

    The loss sum(dO out) is off by r sqrt(sum (dO out)^2 + sum (P dP)^2), r = 2^-8 / sqrt(3), in the mean
    square (the roundings of out and P); a difference of two by sqrt(2) of that, of which four are allowed. A score moves by
    less than 0.2, the third derivative's share is less than 0.2^2 / 6, and the gradients' own rounding is less than that:
    2^-7 of the difference together."""
    q, k, v, dO = _make(12, 1, 2, 1, 90, 200, D, cuda_device, q_scale=0.5)
    out, lse = binding.attend(q, k, v, causal=True)
    grads = binding.attend_backward(q, k, v, out, lse, dO, causal=True)
    S = (q.double() @ k.double().transpose(2, 3)) * D ** -0.5
    P = torch.softmax(S.masked_fill(~oa.visible(90, 200, 200, True, cuda_device), -math.inf), -1)
    dP, G = dO.double() @ v.double().transpose(2, 3), dO.double()
    noise = 2.0 ** -8 / math.sqrt(3) * float((G * (P @ v.double())).square().sum() + (P * dP).square().sum()) ** 0.5
    no_delta = (D ** -0.5 * (P * dP) @ k.double(), (D ** -0.5 * (P * dP).transpose(2, 3) @ q.double()).sum(1, keepdim=True))

    def difference(i, direction):
        d = 2.0 * direction / direction.norm()
        x = (q, k, v)[i].double()
        hi, lo = (x + d).to(torch.bfloat16), (x - d).to(torch.bfloat16)
        val = []
        for x in (hi, lo):
            args = [q, k, v]
            args[i] = x
            val.append(float((binding.attend(*args, causal=True)[0].double() * G).sum()))
        return val[0] - val[1], hi.double() - lo.double()  # the step as bf16 took it

    for i, grad in enumerate(grads):
        got, moved = difference(i, grad.double())
        want = float((grad.double() * moved).sum())
        tol = 4 * math.sqrt(2) * noise + 2.0 ** -7 * abs(want)
        assert tol <= 0.1 * want  # so that no gradient at all, or one of the other sign, would not pass
        assert abs(got - want) <= tol, (i, got, want)
        if i < 2:
            got, moved = difference(i, no_delta[i] - grad.double())
            want, wrong = float((grad.double() * moved).sum()), float((no_delta[i] * moved).sum())
            tol = 4 * math.sqrt(2) * noise + 2.0 ** -7 * abs(want)
            assert abs(got - want) <= tol < abs(got - wrong) / 2, (i, got, want, wrong)
