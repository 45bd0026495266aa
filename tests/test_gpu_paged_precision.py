"""The precision that the interface states for an e4m3 cache: weights and scaled value
rows in fp16 (2^-11 each, three roundings at most), not in bf16."""
import math

import pytest
import torch

from exact_attention_71_gb300 import api
from tests import paged_ref as ref
from tests.test_gpu_paged import SHAPES, Problem
from tests.test_gpu_paged_modes import MODES, shape_id

WEIGHT = 0.5 + 0.98 * 2.0 ** -9      # of every other key: almost between two bf16 numbers


def tolerance(o, spread, delta, weights=3 * 2.0 ** -11):
    """bf16 result (2^-8 of its value), weights and scaled values (`weights` of sum p |v|
    together), scores off by delta (the weights and their sum)."""
    return 2.0 ** -8 * abs(o) + (weights + 2 * delta) * (1 + 2.0 ** -8) * spread


def two_groups(weight):
    """(o, sum p |v|) of as many keys of weight 1 and value 1 as of weight WEIGHT and
    value -2, the latter's weight taken as `weight` in the product."""
    return (1 - 2 * weight) / (1 + WEIGHT), (1 + 2 * WEIGHT) / (1 + WEIGHT)


def bf16(x):
    return float(torch.tensor(x, dtype=torch.float64).to(torch.bfloat16))


def fp16(x):
    return float(torch.tensor(x, dtype=torch.float64).to(torch.float16))


def test_the_two_groups_tell_fp16_weights_from_bf16_ones():
    want, spread = two_groups(WEIGHT)
    tol = tolerance(want, spread, 2.0 ** -17)
    assert abs(two_groups(fp16(WEIGHT))[0] - want) <= tol / 4
    assert abs(two_groups(bf16(WEIGHT))[0] - want) > tol


@pytest.mark.gpu
@pytest.mark.parametrize("segment", ["own", "prefix"])
@pytest.mark.parametrize("kernel, Nq", [("stream", 1), ("stream", 5), ("tile", 40), ("tile", 150)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weights_whose_roundings_add_up(d, kernel, Nq, segment):
    n, ps, H, hkv = 1000, 32, 4, 2
    cache = api.kv_cache(-(-n // ps), ps, hkv, d)
    odd = torch.arange(n, device="cuda") % 2 == 1
    k = torch.zeros((n, hkv, d), dtype=torch.bfloat16, device="cuda")
    k[odd, :, 3] = -1.0
    v = torch.ones_like(k)
    v[odd] = -2.0
    pages = torch.arange(cache.k.shape[0], dtype=torch.int32, device="cuda").flip(0).contiguous()
    at = torch.arange(n, device="cuda")
    api.attn_kv_write(k, v, pages.long()[at // ps] * ps + at % ps, cache)
    q = torch.zeros((1, Nq, H, d), dtype=torch.bfloat16, device="cuda")
    q[..., 3] = 1.0
    scale = -math.log(WEIGHT)
    if segment == "own":
        plan = api.paged_plan(1, Nq, H, hkv, d, 0, len(pages), ps)
        o, lse = api.attn_fwd_paged(q, cache, pages[None], torch.tensor([n], dtype=torch.int32, device="cuda"), causal=False,
                                    scale=scale)
        assert plan.own_kernel == kernel
    else:
        plan = api.paged_plan(1, Nq, H, hkv, d, n, 0, ps)
        o, lse = api.attn_fwd_paged(q, cache, torch.zeros((1, 0), dtype=torch.int32, device="cuda"),
                                    torch.zeros(1, dtype=torch.int32, device="cuda"), pages, n, scale=scale)
        assert plan.prefix_kernel == kernel
    assert api.device_status()[0] == 0
    want, spread = two_groups(WEIGHT)
    # a score is one product of 0.69; its binary32 roundings and exp2's error are below 2^-19
    tol = tolerance(want, spread, 2.0 ** -19)
    assert float((o.double() - want).abs().max()) <= tol
    assert float((lse.double() - math.log(n / 2 * (1 + WEIGHT))).abs().max()) <= 2.0 ** -19


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES + MODES, ids=shape_id)
def test_an_e4m3_cache_is_within_the_stated_precision(shape):
    p = Problem(*shape, fp8=True, seed=81)
    o, lse = p.run()
    assert api.device_status()[0] == 0
    scale = 1.0 / math.sqrt(p.d)
    for b, n in enumerate(p.lens):
        k = torch.cat([p.values("k", -1), p.values("k", b)])
        v = torch.cat([p.values("v", -1), p.values("v", b)])
        sees = [p.prefix + max(0, n - p.Nq + 1 + i) for i in range(p.Nq)]
        q = p.q[b].double()
        want, wl, spread, size = ref.attend(q, k, v, sees)
        if not len(k):
            continue
        # Scores: sums of d products in binary32 (2^-23 of the running magnitude for each
        # addition), three more roundings and exp2 (2^-19); elements of q below 2^-9
        # of their row's largest may be off by 2^-17 of it.
        delta = (p.d + 4) * 2.0 ** -23 * size + 2.0 ** -19
        delta = delta + 2.0 ** -17 * scale * (q.abs().amax(-1) * float(k.abs().sum(-1).max())).transpose(0, 1)
        t = delta.transpose(0, 1)[..., None]
        # Scales far below the largest: 2^-25 of it, and 2^-29 for each key's weight
        # (at most the largest: 1).
        small = (2.0 ** -25 + len(k) * 2.0 ** -29) * float(v.abs().max())
        tol = tolerance(want, spread, t) + small
        assert bool(((o[b].double() - want).abs() <= tol).all()), (b, float(((o[b].double() - want).abs() - tol).max()))
