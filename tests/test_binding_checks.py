"""What the binding and the library refuse before anything is enqueued, where it needs no GPU to see."""

import pytest
import torch

from sparse_linear_attention_sla_b200 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def test_an_output_over_an_expanded_input_is_refused():
    """An input of stride 0 whose memory meets the output's: refused as any overlap is, whichever dimension repeats."""
    buf = torch.zeros(4096, dtype=torch.bfloat16)
    out = buf[:2048].view(1, 4, 8, 64)
    for x in (buf[:512].view(1, 1, 8, 64).expand(1, 4, 8, 64), buf[:64].view(1, 1, 1, 64).expand(1, 4, 8, 64),
              buf[64:320].view(1, 4, 1, 64).expand(1, 4, 8, 64)):
        with pytest.raises(ValueError):
            binding._check_apart("out", out, x)
    apart = buf[2048:2112].view(1, 1, 1, 64).expand(1, 4, 8, 64)
    binding._check_apart("out", out, apart)
    rows = buf.view(1, 1, 32, 128)  # the repeated input lies between the output's rows
    binding._check_apart("out", rows[..., :64], rows[:, :, :1, 64:].expand(1, 1, 32, 64))
