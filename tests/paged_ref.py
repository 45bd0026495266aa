"""Plain 64-bit forms of the paged cache's operators (torch, float64) and their
inputs; no code of the library."""
import math

import torch


def e4m3_round(y):
    """float64 -> nearest e4m3 value, ties to even, saturating at 448."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), y)


def quantise(x):
    """bf16 rows -> (code values, scales) as float64.  The scale and the quotient
    are rounded to float32 first, as the definition says."""
    x32 = x.float()
    amax = x32.abs().amax(-1)
    # (a tensor divisor: torch multiplies by the reciprocal of a Python number)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return e4m3_round((x32 / scale[..., None]).double()), scale


def attend(q, k, v, sees, scale=None):
    """One sequence.  q (Nq, H, d), k and v (L, H_kv, d) float64, sees (Nq,): query
    i sees keys [0, sees[i]).  Returns (o, lse (H, Nq), bound on |o|'s weights
    sum_j p_j |v_j|, largest sum_c |q_c k_jc| * scale)."""
    Nq, H, d = q.shape
    G = H // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    o = torch.zeros_like(q)
    spread = torch.zeros_like(q)
    lse = torch.full((H, Nq), -math.inf, dtype=torch.float64, device=q.device)
    size = torch.zeros((H, Nq), dtype=torch.float64, device=q.device)
    for i in range(Nq):
        n = int(sees[i])
        if n <= 0:
            continue
        s = torch.einsum("hd,jhd->hj", q[i], kk[:n]) * scale
        size[:, i] = (torch.einsum("hd,jhd->hj", q[i].abs(), kk[:n].abs()) * scale).amax(1)
        lse[:, i] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[:, i:i + 1])
        o[i] = torch.einsum("hj,jhd->hd", p, vv[:n])
        spread[i] = torch.einsum("hj,jhd->hd", p, vv[:n].abs())
    return o, lse, spread, size


def tolerances(o, lse, spread, size, d):
    """Elementwise bounds on the kernels' errors.

    A score is a float32 sum of d exact products (each addition off by 2^-23 of
    the running magnitude at most, a truncating accumulator) with three more
    roundings (the scales, the subtraction of the reference), and exp2's own
    error is below 2^-21: a weight is off by at most delta relative, and so is
    their sum.  Each weight is rounded to bf16 once (2^-8), O once more at the end
    (2^-8 of its value); joining partial results adds a few 2^-22.
    """
    delta = (d + 4) * 2.0 ** -23 * size + 2.0 ** -19
    t = delta.transpose(0, 1)[..., None]
    return 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * t) * (1 + 2.0 ** -8) * spread + 1e-30, delta + 2.0 ** -22 * lse.abs()
