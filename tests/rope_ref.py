"""Plain forms of the rotary positions, of trees and of appending to the cache
(torch, float64 or step by step in float32); no code of the library."""
import math

import torch

from tests import paged_ref


def tables(rows, rot, device, base=10000.0):
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def gather(cos, sin, positions, pair_axis, inverse=False):
    """(T, rot / 2) cosines and sines of tokens at positions (axes, T)."""
    at = torch.stack([positions[a] for a in pair_axis], 1)
    return cos.gather(0, at), sin.gather(0, at) * (-1.0 if inverse else 1.0)


def pairs(d, rot, interleaved, device):
    i = torch.arange(rot // 2, device=device)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, c, s, rot, interleaved, dtype=torch.float64):
    """Rows (T, heads, d) turned, in `dtype` (float32: each product and sum rounded).
    Returns (values, sum of the products' magnitudes)."""
    first, second = pairs(x.shape[-1], rot, interleaved, x.device)
    c, s = c[:, None, :].to(dtype), s[:, None, :].to(dtype)
    y = x.to(dtype).clone()
    a, b = y[..., first], y[..., second]
    size = torch.zeros_like(y)
    ac, bs, as_, bc = a * c, b * s, a * s, b * c
    y[..., first], y[..., second] = ac - bs, as_ + bc
    size[..., first], size[..., second] = ac.abs() + bs.abs(), as_.abs() + bc.abs()
    return y, size


def rounding(want, size):
    """Three float32 roundings (2^-24 each, of the products' sizes), one to bf16 (2^-8
    of the value; below bf16's normal range half of its step, 2^-134)."""
    return 2.0 ** -8 * want.abs() + 4 * 2.0 ** -24 * size + 2.0 ** -134


def quantise(x32):
    """float32 rows -> (code values, scales) as the definition says."""
    amax = x32.abs().amax(-1)
    scale = amax / torch.full_like(amax, 448.0)
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return paged_ref.e4m3_round((x32 / scale[..., None]).double()), scale


def paths(parents):
    """parents: a list.  For each node the set of nodes that it sees, or None: no node."""
    n, out = len(parents), []
    for i in range(n):
        seen, at = [], i
        if parents[i] < -1:
            out.append(None)
            continue
        while 0 <= at < n and at not in seen and parents[at] >= -1:
            seen.append(at)
            at = parents[at]
        out.append(set(seen) if at == -1 else None)
    return out


def attend(q, k, v, mask, scale=None):
    """One sequence: q (Nq, H, d), k and v (L, H_kv, d) float64, mask (Nq, L): True
    where the query sees the key.  Returns as paged_ref.attend."""
    Nq, H, d = q.shape
    G = H // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    o, spread = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((H, Nq), -math.inf, dtype=torch.float64, device=q.device)
    size = torch.zeros((H, Nq), dtype=torch.float64, device=q.device)
    for i in range(Nq):
        at = mask[i].nonzero()[:, 0]
        if len(at) == 0:
            continue
        ki, vi = kk[at], vv[at]
        s = torch.einsum("hd,jhd->hj", q[i], ki) * scale
        size[:, i] = (torch.einsum("hd,jhd->hj", q[i].abs(), ki.abs()) * scale).amax(1)
        lse[:, i] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[:, i:i + 1])
        o[i] = torch.einsum("hj,jhd->hd", p, vi)
        spread[i] = torch.einsum("hj,jhd->hd", p, vi.abs())
    return o, lse, spread, size
