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


def _outputs(B, H, N, D):
    """Outputs [B, H, N, D] whose own rows meet (repeated in each dimension, rows that reach into the next), and some
    that do not."""
    at = 1 << 20
    T = binding.Tensor
    meet = [T(at, 0, N * D, D), T(at, H * N * D, 0, D), T(at, H * N * D, N * D, 0), T(at, 0, 0, D), T(at, 0, 0, 0),
            T(at, H * N * D, N * D, D - 8), T(at, H * N * D, (N - 1) * D, D), T(at, (H - 1) * N * D, N * D, D),
            T(at, N * H * D, D - 8, H * D), T(at, N * H * D, D, (H - 1) * D), T(at, 64, 64, 64)]
    apart = [T(at, H * N * D, N * D, D), T(at, N * H * D, D, H * D), T(at, D, B * D, B * H * D), T(at, N * H * (D + 8), D + 8, H * (D + 8)),
             T(at, 1 << 40, 1 << 36, 1 << 30)]
    return meet, apart


# No call here gets as far as a launch: the pointers are none. What comes behind the outputs is missing, and an output
# that is taken shows by the complaint about that.
@pytest.mark.parametrize("B, H, N", [(3, 4, 20), (2, 2, 2)])
def test_rotary_outputs_whose_rows_meet_are_refused(lib, B, H, N):
    D = 64
    spec = binding.rotary_spec((32, 32), grid=(4, 5))
    x = binding.Tensor(1 << 30, H * N * D, N * D, D)

    def says(q, qo, B=B, H=H, N=N):
        both = []
        for call in (lambda: lib.sla_rotary(spec, B, H, H, N, D, 0, q, qo, None, None, None),
                     lambda: lib.sla_rotary_backward(spec, B, H, H, N, D, 1, 1, q, qo, None, None, None)):
            assert call() == 1
            both.append(lib.sla_last_error().decode().split()[0])
        assert both[0] == both[1]
        return both[0]

    meet, apart = _outputs(B, H, N, D)
    for t in meet:
        assert says(x, t) == "q_out" and says(t, t) == "q_out"
        assert says(t, x) == "k"  # as an input it may repeat
        assert lib.sla_rotary(spec, B, H, H, N, D, 0, x, x, x, t, None) == 1
    for t in apart:
        assert says(x, t) == "k" and says(t, t) == "k"
    assert says(x, binding.Tensor(1 << 30, -H * N * D, -N * D, -D)) == "k"
    assert says(x, binding.Tensor(1 << 30, H * N * D, N * D, 8 - D)) == "q_out"
    assert says(x, binding.Tensor(1 << 30, 0, 0, 0), 1, 1, 1) == "k"  # strides that nothing uses


@pytest.mark.parametrize("B, H, N", [(3, 4, 20), (2, 2, 2)])
def test_attention_outputs_whose_rows_meet_are_refused(lib, B, H, N):
    D = 64
    p = binding.AttendProblem(B, H, H, N, N, D, 0, 0.125)
    x = binding.Tensor(1 << 30, H * N * D, N * D, D)
    forward = lambda o: lib.sla_attend(p, x, x, x, None, o, 1 << 21, None, 0, None)  # noqa: E731
    back = lambda *g: lib.sla_attend_backward(p, x, x, x, x, 1 << 21, x, None, *g, None, 0, None)  # noqa: E731
    meet, apart = _outputs(B, H, N, D)
    for t in meet:
        assert forward(t) == 1 and back(t, x, x) == 1 and back(x, t, x) == 1 and back(x, x, t) == 1
    for t in apart[:-1]:  # 3: the workspace is missing
        assert forward(t) == 3 and back(t, x, x) == 3 and back(x, t, x) == 3 and back(x, x, t) == 3


@pytest.mark.gpu
def test_expanded_outputs_are_refused(cuda_device):
    x = torch.randn(2, 3, 10, 64, device=cuda_device).to(torch.bfloat16)
    one = torch.randn(1, 1, 10, 64, device=cuda_device).to(torch.bfloat16)
    wide, kept = one.expand(2, 3, 10, 64), one.clone()
    spec = binding.rotary_spec((64,), grid=(10,))
    rolling = torch.zeros(2 * 3 * 10 * 64, dtype=torch.bfloat16, device=cuda_device).as_strided((2, 3, 10, 64), (1920, 640, 56, 1))
    for f in (lambda: binding.rotary(wide, x, spec, out=(wide, None)), lambda: binding.rotary(x, wide, spec, out=(None, wide)),
              lambda: binding.rotary(x, None, spec, out=(rolling, None)), lambda: binding.attend(x, x, x, out=rolling),
              lambda: binding.rotary_backward(wide, None, spec, out=(wide, None))):
        with pytest.raises((ValueError, binding.SlaError)):
            f()
    assert torch.equal(one, kept) and not rolling.any()
    got = binding.rotary(wide, None, spec)[0]  # as an input it repeats
    assert torch.equal(got, binding.rotary(wide.contiguous(), None, spec)[0])


def test_a_scale_past_fp32_in_base_two_is_refused(lib):
    for scale, status in ((2.3e38, 3), (2.4e38, 1), (3.4e38, 1)):  # 3: the workspace is missing
        p = binding.AttendProblem(1, 2, 2, 8, 8, 64, 0, scale)
        x = binding.Tensor(1 << 30, 2 * 8 * 64, 8 * 64, 64)
        assert (lib.sla_workspace_size_attend(p) > 0) == (status == 3)
        assert lib.sla_attend(p, x, x, x, None, x, 1 << 21, None, 0, None) == status


def test_the_package_gives_every_call_of_rotary_and_attend():
    import sparse_linear_attention_sla_b200 as package

    for name in ("rotary_spec", "rotary", "rotary_backward", "attend", "attend_backward", "attend_problem",
                 "new_workspace_attend", "check"):
        assert getattr(package, name) is getattr(binding, name)
