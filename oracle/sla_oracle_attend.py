"""fp64 reference of dense attention and its gradients (test infrastructure only).

Row by row definition, torch float64 on whatever device the inputs lie:

  s_ij = scale q_i . k_j over the keys that query i sees: j < len_b and, causal,
         j <= i + len_b - Nq
  lse_i = ln sum_j e^(s_ij),  P_ij = e^(s_ij - lse_i),  out_i = sum_j P_ij v_j
  dP = dO V^T,  delta_i = dO_i . out_i,  T = P (dP - delta)
  dQ = scale T K,  dK = scale T^T Q,  dV = P^T dO   (dK, dV summed over a key head's query heads)

A query without keys: out = 0, lse = -inf, zero gradient. Keys behind len_b have zero gradients
and are never read.

``attend`` and ``gradients`` also give, per output element, how far rounding may move it in an
implementation that rounds P, T, out and the results to bf16 once each (half a bf16 step is 2^-8 of the
value) and holds everything else in fp32:

  out: 2^-8 (sum_j P |v_j| + |out|)
  dV:  2^-8 (sum_i P |dO_i| + |dV|)
  dQ:  scale [2^-8 sum_j |T| |k_j| + sum_j P |k_j| e_i] + 2^-8 |dQ|
  dK:  scale [2^-8 sum_i |T| |q_i| + sum_i P |q_i| e_i] + 2^-8 |dK|
       with e_i = 2^-8 sum_d |dO_id| (2 |out_id| + sum_j P |v_jd|), what rounding of P and out
       does to delta_i (which an implementation forms from the rounded out)
  fp32: a score is off by at most (D + 2) 2^-24 scale sum_d |q_d k_d| =: u_i for the worst key that
       row i sees, and lse, rounded itself and then multiplied, by another 2^-23 |lse_i|, so each P by
       2 u_i + 2^-23 |lse_i| + 2^-21 of itself; that factor multiplies the same sums.
  underflow: P and T below 2^-126 (the smallest normal number of bf16 and fp32) may be flushed to
       0, so every P and T is off by another 2^-126 at most, and a result by another 2^-126.

The bounds add every rounding up at its worst, which over many keys is far from what happens. ``norms`` gives
how large the whole error of a result is expected to be: a rounding is off by at most half a step, 2^-8 of the
value, evenly spread, so by at most r = 2^-8 / sqrt(3) of it in the mean square, each on its own:

  out: r^2 [sum_ij P^2 |v_j|^2 + |out|^2]
  dV:  r^2 [sum_ij P^2 |dO_i|^2 + |dV|^2]
  dQ:  scale^2 [r^2 sum_ij T^2 |k_j|^2 + sum_i h_i^2 |sum_j P_ij k_j|^2] + r^2 |dQ|^2
  dK:  scale^2 [r^2 sum_ij T^2 |q_i|^2 + sum_ij h_i^2 P_ij^2 |q_i|^2] + r^2 |dK|^2
       with h_i^2 = r^2 [sum_d (dO_id out_id)^2 + sum_j P_ij^2 dP_ij^2], delta's own error
  fp32: P is off by another 2^-22 (1 + max_j |s_ij| + |lse_i|) of itself in the mean square (the
       additions' roundings go either way), which adds to r^2 for P and T and to h_i.

Parity status: pinned by torch autograd of a masked softmax, by central differences, by
torch's own attention, and by hand values for rows without keys; the bounds and norms by planted mistakes.
"""

from __future__ import annotations

import torch

HALF_STEP = 2.0 ** -8  # of bf16, relative to the value
TINY = 2.0 ** -126     # smallest normal number of bf16 and fp32


def visible(Nq, Nk, n, causal, device):
    j = torch.arange(Nk, device=device)[None, :]
    keep = (j < n).expand(Nq, Nk)
    if causal:
        keep = keep & (j <= torch.arange(Nq, device=device)[:, None] + n - Nq)
    return keep


def _heads(q, k, v, kv_lens, causal, scale):
    """(b, h, key head, q, k[:n], v[:n], P, lse, fp32 factor of the rows [Nq, 1]) of every head."""
    B, H, Nq, D = q.shape
    Hk, Nk = k.shape[1:3]
    lens = [Nk] * B if kv_lens is None else [int(x) for x in kv_lens]
    for b in range(B):
        n = lens[b]
        for h in range(H):
            kh = h // (H // Hk)
            Q, K, V = q[b, h].double(), k[b, kh, :n].double(), v[b, kh, :n].double()
            if n == 0:
                yield (b, h, kh, Q, K, V, torch.zeros(Nq, 0, dtype=torch.float64, device=q.device),
                       torch.full((Nq,), -torch.inf, dtype=torch.float64, device=q.device),
                       torch.zeros(Nq, 1, dtype=torch.float64, device=q.device))
                continue
            S = (Q @ K.T) * scale
            keep = visible(Nq, n, n, causal, q.device)
            S = S.masked_fill(~keep, -torch.inf)
            lse = torch.logsumexp(S, dim=1)
            P = torch.where(lse[:, None] == -torch.inf, 0.0, torch.exp(S - lse[:, None]))
            worst = torch.where(keep, Q.nan_to_num(0.0).abs() @ K.abs().T, 0.0).amax(1) * scale
            size = lse.abs().nan_to_num(posinf=0.0)
            u = 2 * (D + 2) * 2.0 ** -24 * worst + 2.0 ** -23 * size + 2.0 ** -21
            yield b, h, kh, Q, K, V, P, lse, u[:, None]


def attend(q, k, v, kv_lens=None, causal=False, scale=None):
    """(out, lse, bound of out, bound of lse), fp64."""
    D = q.shape[3]
    scale = D ** -0.5 if scale is None else scale
    out, bound = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    lse, lse_bound = (torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device) for _ in range(2))
    for b, h, _, Q, K, V, P, L, u in _heads(q, k, v, kv_lens, causal, scale):
        out[b, h], lse[b, h] = P @ V, L
        bound[b, h] = ((HALF_STEP + u) * P + TINY) @ V.abs() + HALF_STEP * out[b, h].abs() + TINY
        lse_bound[b, h] = u[:, 0] + 2.0 ** -21 * (1 + L.abs().nan_to_num(posinf=0.0))
    return out, lse, bound, lse_bound


def gradients(q, k, v, dO, kv_lens=None, causal=False, scale=None):
    """(dq, dk, dv, and the bound of each), fp64."""
    D = q.shape[3]
    scale = D ** -0.5 if scale is None else scale
    zero = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)  # noqa: E731
    dq, dk, dv, bq, bk, bv = zero(q), zero(k), zero(v), zero(q), zero(k), zero(v)
    for b, h, kh, Q, K, V, P, L, u in _heads(q, k, v, kv_lens, causal, scale):
        n = K.shape[0]
        seen = (L > -torch.inf)[:, None]
        G = torch.where(seen, dO[b, h].double(), 0.0)
        Q = torch.where(seen, Q, 0.0)
        out = P @ V
        delta = (G * out).sum(1)
        dP = G @ V.T
        T = P * (dP - delta[:, None])
        dq[b, h] = scale * (T @ K)
        dk[b, kh, :n] += scale * (T.T @ Q)
        dv[b, kh, :n] += P.T @ G
        e = (HALF_STEP + u) * (G.abs() * (2 * out.abs() + P @ V.abs())).sum(1)[:, None]
        # fp32: dP and delta are off by (D + 2) 2^-24 of their sums of magnitudes, P by u
        fine = P * ((D + 2) * 2.0 ** -24 * (G.abs() @ V.abs().T) + u * (dP.abs() + delta.abs()[:, None]))
        t = HALF_STEP * T.abs() + P * e + fine + TINY * (1 + (dP.abs() + delta.abs()[:, None]))
        bq[b, h] = scale * (t @ K.abs()) + HALF_STEP * dq[b, h].abs() + TINY
        bk[b, kh, :n] += scale * (t.T @ Q.abs())
        bv[b, kh, :n] += ((HALF_STEP + u) * P + TINY).T @ G.abs()
    bk += HALF_STEP * dk.abs() + TINY
    bv += HALF_STEP * dv.abs() + TINY
    return dq, dk, dv, bq, bk, bv


def norms(q, k, v, dO, kv_lens=None, causal=False, scale=None):
    """The expected norms of the errors of out, dq, dk and dv (see above)."""
    D = q.shape[3]
    scale = D ** -0.5 if scale is None else scale
    g = gradients(q, k, v, dO, kv_lens, causal, scale)[:3]
    r2 = HALF_STEP ** 2 / 3
    out2 = dq2 = dk2 = dv2 = 0.0
    for b, h, _, Q, K, V, P, L, _ in _heads(q, k, v, kv_lens, causal, scale):
        if K.shape[0] == 0:
            continue
        seen = (L > -torch.inf)[:, None]
        G = torch.where(seen, dO[b, h].double(), 0.0)
        Q = torch.where(seen, Q, 0.0)
        out, dP = P @ V, G @ V.T
        T = P * (dP - (G * out).sum(1)[:, None])
        S = torch.where(P > 0, (Q @ K.T) * scale, 0.0)
        fine2 = (2.0 ** -22 * (1 + S.abs().amax(1) + L.abs().nan_to_num(posinf=0.0))) ** 2
        w2 = (r2 + fine2)[:, None]
        q2, k2, v2, g2 = ((x * x).sum(1) for x in (Q, K, V, G))
        h2 = r2 * (G * out).square().sum(1) + w2[:, 0] * (P * dP).square().sum(1)
        out2 += float((w2 * P * P @ v2[:, None]).sum() + r2 * out.square().sum())
        dv2 += float((w2 * P * P * g2[:, None]).sum())
        dq2 += scale ** 2 * float((w2 * T * T @ k2[:, None]).sum() + (h2 * (P @ K).square().sum(1)).sum())
        dk2 += scale ** 2 * float(((w2 * T * T + h2[:, None] * P * P) * q2[:, None]).sum())
    own = [r2 * float(x.square().sum()) for x in g]
    return tuple(x ** 0.5 for x in (out2, dq2 + own[0], dk2 + own[1], dv2 + own[2]))
