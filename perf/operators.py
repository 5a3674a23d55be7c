"""The rotary-position and dense-attention operators as cases: their plain forms, the framework's
calls, what each has to read, write and compute, and their values in 64 bits.

Operators:
  rotary        rotation of q and k by positions on one to four axes (time, height, width)
  rotary_back   its transpose, applied to the gradients of the rotated q and k
  attend        softmax(scale q k^T) v with shared key heads, key lengths and a causal mask, and
                the log-sum-exp of every row
  attend_train  attend, then its gradients dq, dk, dv

`own` chooses between the plain form (elementary torch operations in 32 bits, angles in 64) and
the framework's calls.
"""

import math

import torch

own = False

PAIRINGS = {"adjacent": 0, "halves": 1}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # Every denoising step of a Wan2.1-1.3B-shaped model: q and k leave their projections as
        # [B, N, H, D] and the attention wants them rotated, as [B, H, N, D].
        rotary_case("rotary_video", "rotary", 1, 12, 12, 32760, 128, "44,42,42", "21,30,52", layout="bnhd"),
        # Its backward pass: the sparse attention's fp32 gradients, rotated back to bf16 for the
        # projections' gradients.
        rotary_case("rotary_back_video", "rotary_back", 1, 12, 12, 32760, 128, "44,42,42", "21,30,52"),
        # A batch of token sequences of odd length, shared key heads, far positions on one axis.
        rotary_case("rotary_tokens", "rotary", 2, 16, 4, 4093, 64, "64", "", layout="bnhd", pairing="halves",
                    base=1e6, far=1000000),
        # One new token for each of four sequences: latency alone.
        rotary_case("rotary_one_token", "rotary", 4, 12, 12, 1, 128, "44,42,42", "", layout="bnhd", far=1000),
        # The cross attention of the same video model to its text, two prompts of unlike length.
        attend_case("attend_cross", "attend", 2, 12, 12, 32760, 512, 128, lens="512,77", layout="bnhd"),
        # The same, trained.
        attend_case("attend_cross_train", "attend_train", 1, 12, 12, 32760, 512, 128, lens="512"),
        # Dense self attention over an 8192-token sequence, trained: what the sparse attention is
        # tuned against.
        attend_case("attend_self_train", "attend_train", 1, 12, 12, 8192, 8192, 128),
        # Dense self attention over half a video, forward only.
        attend_case("attend_self", "attend", 1, 12, 12, 16380, 16380, 128),
        # Causal training of a token model with shared key heads, D = 64, a ragged length.
        attend_case("attend_causal_train", "attend_train", 2, 16, 4, 2040, 2040, 64, causal=True, layout="bnhd"),
        # One new token for each of four sequences against their keys: bandwidth.
        attend_case("attend_one_token", "attend", 4, 40, 8, 1, 32760, 128, lens="32760,20000,9001,31", causal=True),
        # A chunk of new tokens behind a long prompt.
        attend_case("attend_chunk", "attend", 1, 12, 4, 130, 75600, 128, causal=True),
        # A short sequence, trained: latency.
        attend_case("attend_short_train", "attend_train", 1, 2, 2, 1000, 1000, 128),
    ]


def rotary_case(name, op, B, H, Hk, N, D, axes, grid, layout="bhnd", pairing="adjacent", base=10000.0, far=0):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "N": N, "D": D, "axes": axes, "grid": grid,
            "layout": layout, "pairing": pairing, "base": base, "far": far}


def attend_case(name, op, B, H, Hk, Nq, Nk, D, lens="", causal=False, layout="bhnd"):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "Nq": Nq, "Nk": Nk, "D": D, "lens": lens,
            "causal": causal, "layout": layout}


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_back", "attend", "attend", "attend_train", "attend_train"])
    D = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8, 12])
    H = Hk * rng.choice([1, 1, 2, 4, 5])
    B = rng.choice([1, 1, 2, 3, 4])
    layout = rng.choice(["bhnd", "bnhd"])
    if op.startswith("rotary"):
        # at most what the largest rotary case moves
        N = log_int(rng, 1, max(1, min(32760, 32760 * 24 * 128 // (B * (H + Hk) * D))))
        axes = rng.choice({64: ["64", "24,20,20", "32,32", "16,8"],
                           128: ["128", "44,42,42", "64,64", "32,32,32,32", "96"]}[D])
        n = len(axes.split(","))
        grid = ""
        if rng.random() < 0.5:  # a grid that holds all but a few of the tokens: the rest are not rotated
            side = max(1, int(N ** (1.0 / n)))
            g = [side] * (n - 1)
            g.append(max(1, N // side ** (n - 1)))
            grid = ",".join(str(x) for x in g)
        return rotary_case("", op, B, H, Hk, N, D, axes, grid, layout, rng.choice(["adjacent", "halves"]),
                           rng.choice([10000.0, 1e6]), rng.choice([100, 32768, 1000000]))
    pairs = 8.0e8 if op == "attend_train" else 3.2e9
    Nk = log_int(rng, 1, 32760)
    shape = rng.random()
    causal = rng.random() < 0.4
    if shape < 0.35:
        Nq = Nk
    elif shape < 0.55:
        Nq = rng.choice([1, 2, 5, 17])
    else:
        Nq = log_int(rng, 1, 32760)
    while B * H * Nq * Nk > pairs:
        if Nq >= Nk:
            Nq = Nq * 3 // 4
        else:
            Nk = Nk * 3 // 4
    lens = ""
    if rng.random() < 0.5:
        lens = ",".join(str(rng.choice([Nk, rng.randint(0, Nk), rng.randint(0, Nk)])) for _ in range(B))
    return attend_case("", op, B, H, Hk, Nq, Nk, D, lens, causal, layout)


def numbers(text):
    return [int(x) for x in text.split(",")] if text else []


# ------------------------------------------------------------------------------- inputs

def heads(gen, layout, B, H, N, D, dtype, scale=1.0):
    """[B, H, N, D], laid out so or as a projection leaves it, [B, N, H, D]."""
    shape = (B, N, H, D) if layout == "bnhd" else (B, H, N, D)
    x = (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)
    return x.transpose(1, 2) if layout == "bnhd" else x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, H, Hk, D, layout = case["B"], case["H"], case["Hk"], case["D"], case["layout"]
    state = dict(case)
    if case["op"].startswith("rotary"):
        N = case["N"]
        dtype = torch.float32 if case["op"] == "rotary_back" else torch.bfloat16
        state["q"] = heads(gen, layout, B, H, N, D, dtype)
        state["k"] = heads(gen, layout, B, Hk, N, D, dtype)
        state["axes"] = tuple(numbers(case["axes"]))
        state["grid"] = tuple(numbers(case["grid"]))
        state["positions"] = None
        if not state["grid"]:
            state["positions"] = torch.randint(0, case["far"], (B, N, len(state["axes"])), generator=gen,
                                               device="cuda", dtype=torch.int32)
        return state
    Nq, Nk = case["Nq"], case["Nk"]
    # q and k as a normalised projection leaves them: scores of a few units, a few keys of
    # every row well above the rest.
    state["q"] = heads(gen, layout, B, H, Nq, D, torch.bfloat16, 1.5)
    state["k"] = heads(gen, layout, B, Hk, Nk, D, torch.bfloat16)
    state["v"] = heads(gen, layout, B, Hk, Nk, D, torch.bfloat16)
    lens = numbers(case["lens"])
    state["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    if case["op"] == "attend_train":
        state["dO"] = heads(gen, layout, B, H, Nq, D, torch.bfloat16)
    return state


# ------------------------------------------------------------------------------- plain forms

def token_positions(s, N):
    """[B or 1, N, axes] positions in 64 bits, and which tokens are rotated."""
    if s["positions"] is not None:
        return s["positions"].double(), torch.ones(N, dtype=torch.bool, device="cuda")
    g = s["grid"]
    n = torch.arange(N, device="cuda")
    strides = torch.tensor([math.prod(g[a + 1:]) for a in range(len(g))], device="cuda")
    pos = n[:, None] // strides % torch.tensor(g, device="cuda")
    return pos.double()[None], n < math.prod(g)


def plain_rotary(s, x, sign, dtype):
    N, D = x.shape[2], x.shape[3]
    pos, rotated = token_positions(s, N)
    # for every rotated channel: its axis, its frequency, its partner's channel and the partner's sign
    axis, freq, partner, flip, first = [], [], [], [], 0
    for a, d in enumerate(s["axes"]):
        half = d // 2
        for c in range(d):
            if s["pairing"] == "adjacent":
                i, second, other = c // 2, c % 2, c ^ 1
            else:
                i, second, other = c % half, c // half, (c + half) % d
            axis.append(a)
            freq.append(s["base"] ** (-2.0 * i / d))
            partner.append(first + other)
            flip.append(1.0 if second else -1.0)
        first += d
    dev = x.device
    angle = pos[..., torch.tensor(axis, device=dev)] * torch.tensor(freq, dtype=torch.float64, device=dev)
    cos, sin = angle.cos().float()[:, None], (sign * angle.sin()).float()[:, None]
    xf = x.float()
    head = xf[..., :first]
    turned = head * cos + xf[..., torch.tensor(partner, device=dev)] * torch.tensor(flip, device=dev) * sin
    out = torch.cat([torch.where(rotated[:, None], turned, head), xf[..., first:]], dim=-1)
    return out.to(dtype)


def visible(s):
    """[B or 1, 1, Nq, Nk]: which keys each query sees (None: all)."""
    Nq, Nk = s["Nq"], s["Nk"]
    if s["kv_lens"] is None and not s["causal"]:
        return None
    lens = s["kv_lens"][:, None, None].long() if s["kv_lens"] is not None else torch.full((1, 1, 1), Nk, device="cuda")
    j = torch.arange(Nk, device="cuda")[None, None]
    keep = j < lens
    if s["causal"]:
        i = torch.arange(Nq, device="cuda")[None, :, None]
        keep = keep & (j <= i + lens - Nq)
    return keep[:, None]


def grouped(x, g):
    return x.float().repeat_interleave(g, dim=1) if g > 1 else x.float()


def plain_attend(s):
    """out and lse in 32 bits, and what the gradients need."""
    g = s["H"] // s["Hk"]
    q, k, v = s["q"].float(), grouped(s["k"], g), grouped(s["v"], g)
    scores = q @ k.transpose(-1, -2)
    scores *= s["D"] ** -0.5
    keep = visible(s)
    if keep is not None:
        scores.masked_fill_(~keep, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    scores -= m
    scores.exp_()
    total = scores.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    scores /= torch.where(total == 0, 1.0, total)
    return scores @ v, lse, (q, k, v, scores)


def plain_gradients(s, out, kept):
    g, (q, k, v, p) = s["H"] // s["Hk"], kept
    B, Hk, Nk, D = s["k"].shape
    dO = s["dO"].float()
    dv = p.transpose(-1, -2) @ dO
    ds = dO @ v.transpose(-1, -2)
    ds -= (dO * out).sum(-1, keepdim=True)
    ds *= p
    ds *= s["D"] ** -0.5
    dq = ds @ k
    dk = ds.transpose(-1, -2) @ q
    return dq, dk.view(B, Hk, g, Nk, D).sum(2), dv.view(B, Hk, g, Nk, D).sum(2)


def run(s):
    if s["op"] in ("rotary", "rotary_back"):
        if own:
            from sparse_linear_attention_sla_b200 import binding

            spec = binding.rotary_spec(s["axes"], grid=s["grid"] or None, positions=s["positions"], base=s["base"],
                                       pairing=PAIRINGS[s["pairing"]])
            if s["op"] == "rotary":
                q, k = binding.rotary(s["q"], s["k"], spec)
            else:
                q, k = binding.rotary_backward(s["q"], s["k"], spec, dtype=torch.bfloat16)
        else:
            sign = 1.0 if s["op"] == "rotary" else -1.0
            q, k = plain_rotary(s, s["q"], sign, torch.bfloat16), plain_rotary(s, s["k"], sign, torch.bfloat16)
        return {"q": q, "k": k}
    if own:
        from sparse_linear_attention_sla_b200 import binding

        out, lse = binding.attend(s["q"], s["k"], s["v"], kv_lens=s["kv_lens"], causal=s["causal"])
        if s["op"] == "attend":
            return {"out": out, "lse": lse}
        dq, dk, dv = binding.attend_backward(s["q"], s["k"], s["v"], out, lse, s["dO"], kv_lens=s["kv_lens"],
                                             causal=s["causal"])
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    out, lse, kept = plain_attend(s)
    if s["op"] == "attend":
        return {"out": out.bfloat16(), "lse": lse}
    dq, dk, dv = plain_gradients(s, out, kept)
    return {"out": out.bfloat16(), "lse": lse, "dq": dq.bfloat16(), "dk": dk.bfloat16(), "dv": dv.bfloat16()}


# ------------------------------------------------------------------------------- work

def work(case):
    B, H, Hk, D = case["B"], case["H"], case["Hk"], case["D"]
    if case["op"].startswith("rotary"):
        n = B * (H + Hk) * case["N"]
        read = 4 if case["op"] == "rotary_back" else 2
        positions = 0 if case["grid"] else 4 * B * case["N"] * len(numbers(case["axes"]))
        return {"bytes": n * D * (read + 2) + positions, "flops": 3 * n * sum(numbers(case["axes"]))}
    Nq, Nk = case["Nq"], case["Nk"]
    pairs, keys = 0, 0
    for n in numbers(case["lens"]) or [Nk] * B:
        keys += n
        if case["causal"]:  # query i sees max(0, i + n - Nq + 1) keys
            low = max(0, n - Nq + 1)
            rows = n - low + 1 if n else 0
            pairs += (low + n) * rows // 2
        else:
            pairs += Nq * n
    pairs *= H
    q, kv = 2 * B * H * Nq * D, 2 * Hk * keys * D
    forward = {"bytes": 2 * q + 2 * kv + 4 * B * H * Nq, "flops": 4 * pairs * D}
    if case["op"] == "attend":
        return forward
    # the backward pass reads q, k, v, out, dO and lse and writes dq, dk, dv
    return {"bytes": forward["bytes"] + 4 * q + 2 * kv + 4 * B * H * Nq + 4 * B * Hk * Nk * D,
            "flops": 14 * pairs * D}


# ------------------------------------------------------------------------------- in 64 bits

def exact_rotary(s, x, direction):
    """Each pair as a complex number times e^(i angle), token by token position."""
    N = x.shape[2]
    out = x.double().clone()
    for b in range(x.shape[0]):
        if s["positions"] is not None:
            pos, upto = s["positions"][b].double(), N
        else:
            upto = min(N, math.prod(s["grid"]))
            pos = torch.cartesian_prod(*[torch.arange(g, device=x.device) for g in s["grid"]])
            pos = pos.reshape(-1, len(s["grid"]))[:upto].double()
        at = 0
        for a, d in enumerate(s["axes"]):
            theta = torch.exp(-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d * math.log(s["base"]))
            turn = torch.polar(torch.ones_like(pos[:, a:a + 1] * theta), direction * pos[:, a:a + 1] * theta)
            if s["pairing"] == "adjacent":
                one, two = slice(at, at + d, 2), slice(at + 1, at + d, 2)
            else:
                one, two = slice(at, at + d // 2), slice(at + d // 2, at + d)
            z = torch.complex(x[b, :, :upto, one].double(), x[b, :, :upto, two].double()) * turn
            out[b, :, :upto, one], out[b, :, :upto, two] = z.real, z.imag
            at += d
    return out


def exact_attend(s):
    """Head by head over the keys that each sequence has, every row from its own keys."""
    B, H, Nq, D = s["q"].shape
    Hk, Nk = s["k"].shape[1:3]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    r = {"out": torch.zeros(B, H, Nq, D, **f64), "lse": torch.full((B, H, Nq), -math.inf, **f64)}
    train = "dO" in s
    if train:
        r.update(dq=torch.zeros(B, H, Nq, D, **f64), dk=torch.zeros(B, Hk, Nk, D, **f64),
                 dv=torch.zeros(B, Hk, Nk, D, **f64))
    lens = s["kv_lens"].tolist() if s["kv_lens"] is not None else [Nk] * B
    for b in range(B):
        n = lens[b]
        first = max(0, Nq - n) if s["causal"] else 0  # rows before it see no key
        if n == 0 or first >= Nq:
            continue
        for h in range(H):
            kh = h * Hk // H
            q, k, v = s["q"][b, h, first:].double(), s["k"][b, kh, :n].double(), s["v"][b, kh, :n].double()
            x = torch.matmul(q, k.t()) / math.sqrt(D)
            if s["causal"]:
                x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu_(n - Nq + first + 1), -math.inf)
            lse = torch.logsumexp(x, dim=1)
            p = torch.exp(x - lse[:, None])
            del x
            o = torch.matmul(p, v)
            r["out"][b, h, first:], r["lse"][b, h, first:] = o, lse
            if train:
                dO = s["dO"][b, h, first:].double()
                r["dv"][b, kh, :n] += torch.matmul(p.t(), dO)
                t = p * (torch.matmul(dO, v.t()) - torch.einsum("nd,nd->n", dO, o)[:, None]) / math.sqrt(D)
                r["dq"][b, h, first:] = torch.matmul(t, k)
                r["dk"][b, kh, :n] += torch.matmul(t.t(), q)
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        direction = 1.0 if case["op"] == "rotary" else -1.0
        return {"q": exact_rotary(s, s["q"], direction), "k": exact_rotary(s, s["k"], direction)}
    return exact_attend(s)
