"""GPU parity of dense attention (attend, attend_backward) against the fp64 oracle.

Tolerances are the oracle's per-element bounds: one rounding to bf16 (half a step, 2^-8) each of P, T, out
and the results, and fp32 everywhere else.
"""

import math

import pytest
import torch

from oracle import sla_oracle_attend as oa
from sparse_linear_attention_sla_b200 import binding

pytestmark = pytest.mark.gpu


def _make(seed, B, H, Hk, Nq, Nk, D, dev, layout="bhnd", q_scale=1.5):
    g = torch.Generator(device=dev).manual_seed(seed)

    def one(h, n, s=1.0):
        shape = (B, n, h, D) if layout == "bnhd" else (B, h, n, D)
        x = (torch.randn(shape, generator=g, device=dev) * s).to(torch.bfloat16)
        return x.transpose(1, 2) if layout == "bnhd" else x

    return one(H, Nq, q_scale), one(Hk, Nk), one(Hk, Nk), one(H, Nq)


def _within(name, got, ref, bound):
    got = got.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - bound
    worst = float(over.max())
    assert worst <= 0, f"{name}: {worst:.3e} beyond its bound at {int(over.argmax())}"


def _check(q, k, v, dO, lens=None, causal=False, scale=None, backward=True):
    dev = q.device
    kv = torch.tensor(lens, dtype=torch.int32, device=dev) if lens is not None else None
    p = binding.attend_problem(q, k, causal, scale)
    ws = binding.new_workspace_attend(p, dev)
    out, lse = binding.attend(q, k, v, kv, causal, scale, ws=ws)
    binding.check(ws)
    ref, rlse, bound, lbound = oa.attend(q, k, v, lens, causal, scale)
    _within("out", out, ref, bound)
    dead = rlse == -math.inf
    assert torch.equal(lse == -math.inf, dead)
    assert (out[dead] == 0).all()
    _within("lse", lse.masked_fill(dead, 0.0), rlse.masked_fill(dead, 0.0), lbound)
    if not backward:
        return out, lse
    ws = binding.new_workspace_attend(p, dev, backward=True)
    got = binding.attend_backward(q, k, v, out, lse, dO, kv, causal, scale, ws=ws)
    binding.check(ws)
    refs = oa.gradients(q, k, v, dO, lens, causal, scale)
    for i, name in enumerate(("dq", "dk", "dv")):
        _within(name, got[i], refs[i], refs[i + 3])
    return (out, lse) + got


SHAPES = [
    # B, H, Hk, Nq, Nk
    (1, 1, 1, 128, 128),
    (1, 2, 2, 1, 1),
    (1, 2, 1, 1, 300),
    (2, 3, 3, 77, 513),
    (1, 2, 2, 257, 64),
    (2, 4, 2, 300, 300),
    (1, 6, 2, 129, 1000),
    (1, 2, 2, 1000, 1000),
    (3, 5, 1, 33, 2049),
    (1, 1, 1, 2500, 129),
    (2, 10, 2, 13, 1500),   # nine heads of thirteen queries to a tile: five fit
    (1, 24, 2, 11, 700),    # twelve heads of a group: eleven in one tile, one in the next
    (1, 3, 3, 128, 777),    # the most queries of one tile
    (40, 4, 2, 130, 130),   # more units than SMs
    (2, 6, 2, 130, 700),    # tiles of three heads and 42 queries
    (2, 40, 40, 500, 500),  # causal: whole units, longest first, in waves of both directions
    (3, 36, 12, 700, 650),  # the same with more queries than keys and shared key heads
    (1, 10, 2, 200, 333),   # tiles of five heads and 25 queries where that makes fewest, or equally many and causal
]


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matches_oracle(cuda_device, shape, causal, D):
    B, H, Hk, Nq, Nk = shape
    q, k, v, dO = _make(Nq * 7 + Nk, B, H, Hk, Nq, Nk, D, cuda_device)
    _check(q, k, v, dO, causal=causal)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq, Nk, lens", [
    (200, 300, [300, 0, 1]), (64, 500, [127, 128, 129]), (300, 200, [200, 5, 130]), (1, 4000, [4000, 31, 2600]),
    (1, 5, [0, 0, 0]), (700, 700, [700, 383, 256]),
])
def test_lengths_and_padding(cuda_device, Nq, Nk, lens, causal, D):
    """Keys behind a length hold NaN and infinities; queries that see no key hold NaN."""
    q, k, v, dO = _make(Nq + Nk, 3, 4, 2, Nq, Nk, D, cuda_device, layout="bnhd")
    for b, n in enumerate(lens):
        k[b, :, n:] = math.nan
        v[b, :, n::2], v[b, :, n + 1::2] = math.inf, math.nan
        dead = Nq if n == 0 else max(0, Nq - n) if causal else 0
        q[b, :, :dead] = math.nan
        dO[b, :, :dead] = math.nan
    _, _, dq, dk, dv = _check(q, k, v, dO, lens, causal)
    for b, n in enumerate(lens):
        assert (dk[b, :, n:] == 0).all() and (dv[b, :, n:] == 0).all()


@pytest.mark.parametrize("D", [128, 64])
def test_moving_reference(cuda_device, D):
    """Row maxima that grow from tile to tile by tens and by thousands, and fall."""
    q, k, v, dO = _make(3, 1, 2, 2, 200, 1100, D, cuda_device)
    ramp = torch.linspace(0.02, 12, 1100, device=cuda_device)
    up = (k * ramp[None, None, :, None]).to(torch.bfloat16)
    _check(q, up, v, dO)
    _check(q, up.flip(2).contiguous(), v, dO)
    _check((q * 40).to(torch.bfloat16), up, v, dO)
    first = k.clone()
    first[:, :, :128] *= -60  # the first tile far above or below the rest
    _check(q, first, v, dO)


def test_scores_near_the_end_of_the_range(cuda_device):
    """Scores of 1e38, whose rounding alone passes what an exponential can hold: whatever comes out, it comes, and the
    other rows are as they are without it."""
    q, k, v, dO = _make(14, 1, 2, 2, 140, 300, 128, cuda_device)
    want, wlse = binding.attend(q, k, v)
    big = q.clone()
    big[:, :, 7] = 3e37
    p = binding.attend_problem(big, k)
    ws = binding.new_workspace_attend(p, cuda_device)
    out, lse = binding.attend(big, k, v, ws=ws)
    binding.check(ws)
    keep = torch.arange(140, device=cuda_device) != 7
    assert torch.equal(out[:, :, keep], want[:, :, keep]) and torch.equal(lse[:, :, keep], wlse[:, :, keep])
    for Nq in (1, 40):  # one tile, most of whose rows are no query
        ws = binding.new_workspace_attend(binding.attend_problem(big[:, :, 7:7 + Nq], k), cuda_device)
        out, _ = binding.attend(big[:, :, 7:7 + Nq], k, v, ws=ws)
        binding.check(ws)
        assert torch.equal(out[:, :, 1:], binding.attend(q[:, :, 7:7 + Nq], k, v)[0][:, :, 1:])


def test_scale(cuda_device):
    q, k, v, dO = _make(9, 1, 2, 2, 150, 333, 128, cuda_device)
    for scale in (1e-4, 0.5):
        _check(q, k, v, dO, scale=scale)


def test_layouts_and_outputs(cuda_device):
    """Slices of one packed projection, and out written into a strided view."""
    dev = cuda_device
    B, N, H, D = 2, 210, 3, 128
    g = torch.Generator(device=dev).manual_seed(1)
    packed = torch.randn(B, N, 3, H, D + 8, generator=g, device=dev).to(torch.bfloat16)
    q, k, v = (packed[:, :, i, :, 8:].transpose(1, 2) for i in range(3))
    dO = torch.randn(B, N, H, D, generator=g, device=dev).to(torch.bfloat16).transpose(1, 2)
    got = _check(q, k, v, dO)
    plain = _check(q.contiguous(), k.contiguous(), v.contiguous(), dO.contiguous())
    for a, b in zip(got, plain):
        assert torch.equal(a, b)
    room = torch.full((B, N + 3, H, D), 7.0, dtype=torch.bfloat16, device=dev)
    out, lse = binding.attend(q, k, v, out=room[:, 2:N + 2].transpose(1, 2))
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
    assert (room[:, :2] == 7).all() and (room[:, N + 2:] == 7).all()
    odd = torch.zeros(B * H * N * D + 8, dtype=torch.bfloat16, device=dev)[8:].view(B, H, N, D)  # 16-byte rows
    out, _ = binding.attend(q, k, v, out=odd)
    assert torch.equal(out, got[0])


@pytest.mark.parametrize("Nq, Nk, lens", [(300, 2, None), (40, 3, None), (257, 128, None), (300, 700, [2, 1, 5])])
@pytest.mark.parametrize("D", [128, 64])
def test_gradients_of_few_keys(cuda_device, Nq, Nk, lens, D):
    """delta of few keys is formed from P and dP, not from the rounded out. What is left are two roundings to bf16
    (T, then the result), off by at most 2^-8 each and, evenly spread over a step of 2^-7 to 2^-8 of the
    value, by less than 2^-8 / sqrt(3) in the mean square: less than 2^-8 sqrt(2 / 3) of the norm together."""
    q, k, v, dO = _make(Nq + Nk, 3, 4, 2, Nq, Nk, D, cuda_device)
    _, _, dq, dk, _ = _check(q, k, v, dO, lens)
    refs = oa.gradients(q, k, v, dO, lens)
    for got, ref in ((dq, refs[0]), (dk, refs[1])):
        assert float((got.double() - ref).norm() / ref.norm()) <= 2.0 ** -8 * math.sqrt(2 / 3)


def test_causal_dq_of_first_queries(cuda_device):
    """The first 128 queries of a causal sequence have their delta from P and dP: their dq is the one that they have
    alone, within the roundings of T and of dq itself (see test_gradients_of_few_keys). Row 0 sees one key: its
    dq is 0 but for rounding."""
    q, k, v, dO = _make(5, 1, 2, 1, 400, 400, 128, cuda_device)
    out, lse = binding.attend(q, k, v, causal=True)
    dq = binding.attend_backward(q, k, v, out, lse, dO, causal=True)[0]
    s = lambda x, n: x[:, :, :n].contiguous()  # noqa: E731
    short = binding.attend_backward(s(q, 128), s(k, 128), s(v, 128), s(out, 128), s(lse, 128), s(dO, 128), causal=True)[0]
    assert torch.equal(dq[:, :, :128], short)
    ref = oa.gradients(q, k, v, dO, causal=True)[0][:, :, 1:128]
    assert (dq[:, :, 1:128].double() - ref).norm() <= 2.0 ** -8 * math.sqrt(2 / 3) * ref.norm()


def test_nan_gradients_stay_out_of_rows_without_a_part(cuda_device):
    """NaN in dO spreads to what it enters; keys behind a length and queries without keys get exact zeros."""
    for Nq, Nk, n, causal in ((40, 300, 130, False), (300, 200, 60, True)):
        q, k, v, dO = _make(1, 1, 4, 2, Nq, Nk, 128, cuda_device)
        lens = torch.tensor([n], dtype=torch.int32, device=cuda_device)
        out, lse = binding.attend(q, k, v, lens, causal=causal)
        dO = torch.full_like(dO, math.nan)
        k[:, :, n - 1] = math.nan  # a key of the sequence
        dq, dk, dv = binding.attend_backward(q, k, v, out, lse, dO, lens, causal=causal)
        assert (dk[:, :, n:] == 0).all() and (dv[:, :, n:] == 0).all()
        dead = max(0, Nq - n) if causal else 0
        assert (dq[:, :, :dead] == 0).all() and dq[:, :, dead:].isnan().all()
        assert dv[:, :, :n].isnan().all()


def test_equal_calls_give_equal_bits(cuda_device):
    for Nq, Nk in ((1, 3000), (640, 640)):
        q, k, v, dO = _make(5, 2, 4, 2, Nq, Nk, 128, cuda_device)
        a, b = (_check(q, k, v, dO, causal=True) for _ in range(2))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_lengths_outside_are_reported(cuda_device):
    q, k, v, dO = _make(6, 3, 2, 2, 40, 150, 128, cuda_device)
    lens = torch.tensor([-3, 151, 77], dtype=torch.int32, device=cuda_device)
    p = binding.attend_problem(q, k)
    ws = binding.new_workspace_attend(p, cuda_device)
    out, _ = binding.attend(q, k, v, lens, ws=ws)
    with pytest.raises(binding.SlaError) as e:
        binding.check(ws)
    assert e.value.status == 7
    binding.check(ws)  # cleared
    want, _ = binding.attend(q, k, v, lens.clamp(0, 150))
    assert torch.equal(out, want)


def test_gradients_against_differences(cuda_device):
    """Directional differences of the kernel's own forward, summed in fp64.

    The loss sum(dO out) has n = B H Nq D terms, each off by at most its bound of about
    2^-8 (|out| + sum P |v|); with independent signs the difference quotient over 2 h is off by about
    2^-8 sqrt(2 sum (dO bound)^2) / (2 h); five of those are allowed, and h^2 for the third derivative."""
    dev = cuda_device
    q, k, v, dO = _make(12, 1, 2, 1, 90, 200, 128, dev, q_scale=0.5)
    out, lse = binding.attend(q, k, v, causal=True)
    grads = binding.attend_backward(q, k, v, out, lse, dO, causal=True)
    bound = oa.attend(q, k, v, None, True)[2]
    noise = float((dO.double() * bound).square().sum().mul(2).sqrt())
    g = torch.Generator(device=dev).manual_seed(2)
    xs = [q, k, v]
    for i, h in ((0, 2.0 ** -3), (1, 2.0 ** -3), (2, 2.0 ** -3)):
        step = torch.randn(xs[i].shape, generator=g, device=dev)
        hi, lo = (xs[i].float() + h * step).to(torch.bfloat16), (xs[i].float() - h * step).to(torch.bfloat16)
        moved = (hi.double() - lo.double()) / (2 * h)  # the step as bf16 took it
        val = []
        for x in (hi, lo):
            args = list(xs)
            args[i] = x
            val.append(float((binding.attend(*args, causal=True)[0].double() * dO.double()).sum()))
        got = (val[0] - val[1]) / (2 * h)
        want = float((grads[i].double() * moved).sum())
        size = float((grads[i].double().square() * moved.square()).sum().sqrt())
        assert abs(got - want) <= 5 * noise / (2 * h) + 4 * h * h * size + 2.0 ** -8 * 5 * size, (i, got, want)


def test_captured_and_replayed(cuda_device):
    dev = cuda_device
    q, k, v, dO = _make(21, 1, 4, 2, 1, 2000, 128, dev)
    Q, K, V, G = _make(22, 1, 2, 2, 260, 260, 64, dev)
    s = torch.cuda.Stream(dev)
    with torch.cuda.stream(s):
        for _ in range(2):
            binding.attend_backward(Q, K, V, *binding.attend(Q, K, V, causal=True), G, causal=True)
            binding.attend(q, k, v)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o1, l1 = binding.attend(q, k, v)
        o2, l2 = binding.attend(Q, K, V, causal=True)
        g2 = binding.attend_backward(Q, K, V, o2, l2, G, causal=True)
    for seed in (31, 32):
        for dst, src in zip((q, k, v), _make(seed, 1, 4, 2, 1, 2000, 128, dev)):
            dst.copy_(src)
        for dst, src in zip((Q, K, V, G), _make(seed + 5, 1, 2, 2, 260, 260, 64, dev)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize(dev)
        assert torch.equal(o1, binding.attend(q, k, v)[0])
        want = _check(Q, K, V, G, causal=True)
        for a, b in zip((o2, l2) + g2, want):
            assert torch.equal(a, b)


def test_streams_run_side_by_side(cuda_device):
    dev = cuda_device
    data = [_make(40 + i, 1, 2, 2, 500, 700, 128, dev) for i in range(3)]
    want = [binding.attend(q, k, v) for q, k, v, _ in data]
    torch.cuda.synchronize(dev)
    streams = [torch.cuda.Stream(dev) for _ in data]
    got = []
    for s, (q, k, v, dO) in zip(streams, data):
        with torch.cuda.stream(s):
            o, l = binding.attend(q, k, v)
            got.append((o, l, binding.attend_backward(q, k, v, o, l, dO)))
    torch.cuda.synchronize(dev)
    for (o, l, grads), (wo, wl), (q, k, v, dO) in zip(got, want, data):
        assert torch.equal(o, wo) and torch.equal(l, wl)
        for a, b in zip(grads, binding.attend_backward(q, k, v, wo, wl, dO)):
            assert torch.equal(a, b)


def test_refusals(cuda_device):
    q, k, v, dO = _make(1, 1, 4, 2, 20, 30, 128, cuda_device)
    out, lse = binding.attend(q, k, v)
    bad = [
        lambda: binding.attend(q.float(), k, v),
        lambda: binding.attend(q, k, v[:, :, :29]),
        lambda: binding.attend(q[:, :3], k, v),                       # 3 heads over 2
        lambda: binding.attend(q, k[:, :1].expand(1, 2, 30, 128), v),  # stride 0
        lambda: binding.attend(q[..., :96], k[..., :96], v[..., :96]),
        lambda: binding.attend(q, k, v, scale=0.0),
        lambda: binding.attend(q, k, v, scale=math.nan),
        lambda: binding.attend(q, k, v, kv_lens=torch.ones(1, device=cuda_device)),
        lambda: binding.attend(q.cpu(), k, v),
        lambda: binding.attend(q[:, :, :0], k, v),
        lambda: binding.attend(q.transpose(2, 3).contiguous().transpose(2, 3), k, v),
        lambda: binding.attend(q, k, v, ws=torch.empty(64, dtype=torch.uint8, device=cuda_device)),
        lambda: binding.attend(q, k, v, ws=torch.empty(1 << 24, dtype=torch.uint8)),                           # on the host
        lambda: binding.attend(q, k, v, ws=torch.empty(1 << 22, dtype=torch.float32, device=cuda_device)),
        lambda: binding.attend_backward(q, k, v, out, lse, dO, ws=torch.empty(1 << 24, dtype=torch.uint8)),
        lambda: binding.attend(q, k, v, out=q),
        lambda: binding.attend_backward(q, k, v, out, lse.double(), dO),
        lambda: binding.attend_backward(q, k, v, out, lse, dO[:, :, 1:]),
    ]
    for f in bad:
        with pytest.raises((ValueError, binding.SlaError)):
            f()
    _check(q, k, v, dO)
