"""Rotary positions of bf16 q and k (attn_rope), forward and transposed, against
64-bit forms."""
import math

import pytest
import torch

from exact_attention_71_gb300 import api
from tests import rope_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def sections(half, axes, mixed):
    if mixed:
        return tuple(i % axes for i in range(half))
    return tuple(min(i * axes // half, axes - 1) for i in range(half))


def check(got, x, cos, sin, positions, pair_axis, rot, interleaved, inverse=False):
    c, s = ref.gather(cos, sin, positions, pair_axis, inverse)
    want, size = ref.turn(x, c, s, rot, interleaved)
    err = (got.double() - want).abs()
    within = bool((err <= ref.rounding(want, size)).all())
    assert within, float(err.max())
    assert torch.equal(got[..., rot:], x[..., rot:])


# tokens, H, H_kv, d, rot, axes, alternating, interleaved: both numbers of heads a
# lane, heads that do not fill a lane's, one axis and several, sections that end
# inside four pairs, a part of the head.
CASES = [
    (1, 1, 1, 64, 64, 1, False, False),
    (1, 8, 2, 128, 128, 3, False, True),
    (37, 3, 1, 64, 32, 2, False, False),
    (130, 7, 5, 128, 112, 3, True, False),
    (129, 4, 4, 256, 256, 1, False, True),
    (75, 6, 2, 256, 64, 4, True, True),
    (33, 2, 2, 64, 16, 1, False, True),
    (50, 5, 3, 128, 96, 4, False, False),
    (5003, 9, 3, 128, 128, 1, False, False),
    (4099, 13, 3, 128, 128, 3, False, False),
    (9001, 5, 2, 64, 48, 2, True, True),
    (2500, 11, 6, 256, 240, 3, False, False),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_rows_are_turned_by_their_positions(case, inverse):
    T, H, hkv, d, rot, axes, mixed, il = case
    g = gen(1)
    q, k = rand(g, T, H, d), rand(g, T, hkv, d)
    cos, sin = ref.tables(4001, rot, DEV)
    pos = torch.randint(0, 4001, (axes, T), generator=g, device=DEV)
    pair_axis = sections(rot // 2, axes, mixed)
    a, b = api.attn_rope(q, k, cos, sin, pos if axes > 1 else pos[0], pair_axis if axes > 1 else None, il, inverse)
    assert api.device_status()[0] == 0
    check(a, q, cos, sin, pos, pair_axis, rot, il, inverse)
    check(b, k, cos, sin, pos, pair_axis, rot, il, inverse)


@pytest.mark.parametrize("B,N", [(3, 70), (2, 2100)])
def test_batches_share_positions_or_have_their_own(B, N):
    g = gen(2)
    H, hkv, d = 6, 2, 128
    x = rand(g, B, N, H + 2 * hkv, d)                                     # columns of a projection
    q, k = x[:, :, :H], x[:, :, H:H + hkv]
    cos, sin = ref.tables(N + 9, d, DEV)
    n = torch.arange(N, device=DEV)
    own = torch.randint(0, N, (B, N), generator=g, device=DEV)
    flat = lambda t: t.reshape(B * N, -1, d)
    for given, pos in ((None, n.repeat(B)), (n + 9 - 1, (n + 9 - 1).repeat(B)), (own, own.flatten())):
        a, b = api.attn_rope(q, k, cos, sin, given)
        check(flat(a), flat(q), cos, sin, pos[None], (0,) * (d // 2), d, False)
        check(flat(b), flat(k), cos, sin, pos[None], (0,) * (d // 2), d, False)
    # several axes, shared and not
    pair_axis = sections(d // 2, 2, False)
    shared = torch.stack([n // 7, n % 7])
    many = torch.randint(0, N, (2, B, N), generator=g, device=DEV)
    for given, pos in ((shared, shared.repeat(1, B)), (many, many.flatten(1))):
        a, b = api.attn_rope(q, k, cos, sin, given, pair_axis)
        check(flat(a), flat(q), cos, sin, pos, pair_axis, d, False)
        check(flat(b), flat(k), cos, sin, pos, pair_axis, d, False)
    assert api.device_status()[0] == 0


@pytest.mark.parametrize("T", [5, 6000])
def test_in_place_without_k_and_strided_outputs(T):
    g = gen(3)
    H, hkv, d, rot = 5, 2, 64, 32
    cos, sin = ref.tables(T, rot, DEV)
    x = rand(g, T, H + hkv + 1, d)
    q, k = x[:, :H].contiguous(), x[:, H:H + hkv].contiguous()
    want = api.attn_rope(q, k, cos, sin)
    alone, none = api.attn_rope(q, None, cos, sin)
    assert none is None and torch.equal(alone, want[0])
    buf = torch.full((T, 2 * (H + hkv), d), 7.0, dtype=torch.bfloat16, device=DEV)
    a, b = api.attn_rope(x[:, :H], x[:, H:H + hkv], cos, sin, out_q=buf[:, 1:1 + H], out_k=buf[:, 8:8 + hkv])
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    rest = torch.ones(buf.shape[1], dtype=torch.bool)
    rest[1:1 + H] = rest[8:8 + hkv] = False
    assert bool((buf[:, rest] == 7.0).all())
    last = x[:, -1].clone()
    api.attn_rope(x[:, :H], x[:, H:H + hkv], cos, sin, out_q=x[:, :H], out_k=x[:, H:H + hkv])
    assert torch.equal(x[:, :H], want[0]) and torch.equal(x[:, H:H + hkv], want[1]) and torch.equal(x[:, -1], last)


def test_far_positions_and_large_tables():
    """A table of more than 2^31 bytes; positions near its end."""
    rows, d = (1 << 22) + 5, 256
    cos, sin = torch.empty((rows, d // 2), device=DEV), torch.empty((rows, d // 2), device=DEV)
    c, s = ref.tables(64, d, DEV)
    cos[-64:], sin[-64:] = c, s
    q = rand(gen(4), 64, 2, d)
    pos = rows - 64 + torch.arange(64, device=DEV)
    got, _ = api.attn_rope(q, None, cos, sin, pos)
    want, _ = api.attn_rope(q, None, c, s)
    assert torch.equal(got, want) and api.device_status()[0] == 0


@pytest.mark.parametrize("T", [9, 6000])
def test_positions_outside_the_tables_give_rows_of_zeros_and_are_reported(T):
    g = gen(5)
    q, k = rand(g, T, 6, 128), rand(g, T, 2, 128)
    cos, sin = ref.tables(T, 128, DEV)
    pos = torch.arange(T, device=DEV).repeat(2, 1)
    pair_axis = sections(64, 2, False)
    want = api.attn_rope(q, k, cos, sin, pos, pair_axis)
    pos[1, 2], pos[0, 5], pos[1, 7] = T, -1, 1 << 60
    got = api.attn_rope(q, k, cos, sin, pos, pair_axis)
    assert api.device_status() == (-5, 0x104) and api.device_status()[0] == 0
    for a, b in zip(got, want):
        b[[2, 5, 7]] = 0.0
        assert torch.equal(a, b)


def test_infinities_stay_in_their_pair():
    q = rand(gen(6), 3, 2, 64)
    q[1, 0, 5] = INF
    q[2, 1, 40] = NAN                      # past the 32 that turn
    cos, sin = ref.tables(3, 32, DEV)
    for il in (False, True):
        got, _ = api.attn_rope(q, None, cos, sin, interleaved=il)
        bad = ~torch.isfinite(got)
        first, second = ref.pairs(64, 32, il, DEV)
        pair = int(((first == 5) | (second == 5)).nonzero()[0])
        where = {(1, 0, int(first[pair])), (1, 0, int(second[pair])), (2, 1, 40)}
        assert {tuple(x) for x in bad.nonzero().tolist()} == where


def test_the_gradient_of_attention_behind_the_rotation():
    """attn_rope, attn_fwd, attn_bwd, attn_rope(inverse): against float64 autograd and
    central differences.  The rotated q and k, and the gradient, are rounded to bf16
    (2^-8 of a value each), beside the backward's own 5e-3 (relative RMS)."""
    B, N, H, hkv, d, rot = 1, 150, 4, 2, 64, 48
    tol = 5e-3 + 3 * 2.0 ** -8
    g = gen(7)
    q, k, v, do = rand(g, B, N, H, d), rand(g, B, N, hkv, d), rand(g, B, N, hkv, d), rand(g, B, N, H, d)
    cos, sin = ref.tables(40, rot, DEV)
    n = torch.arange(N, device=DEV)
    pos, pair_axis = torch.stack([n // 36, n // 6 % 6, n % 6]), sections(rot // 2, 3, True)
    q1, k1 = api.attn_rope(q, k, cos, sin, pos, pair_axis)
    o, lse = api.attn_fwd(q1, k1, v, causal=True)
    dq1, dk1, dv = api.attn_bwd(do, q1, k1, v, o, lse, causal=True)
    dq, dk = api.attn_rope(dq1, dk1, cos, sin, pos, pair_axis, inverse=True)
    torch.cuda.synchronize()
    c, s = ref.gather(cos, sin, pos, pair_axis)

    def loss(qq, kk, vv):
        a, b = ref.pairs(d, rot, False, DEV)
        def turned(x):
            y = x[..., :rot]
            lo, hi = y[..., a], y[..., b]
            cc, ss = c[:, None].double(), s[:, None].double()
            return torch.cat([lo * cc - hi * ss, lo * ss + hi * cc, x[..., rot:]], -1)
        qt, kt = turned(qq[0]), turned(kk[0]).repeat_interleave(H // hkv, 1)
        sc = torch.einsum("ihd,jhd->hij", qt, kt) / math.sqrt(d)
        sc = sc.masked_fill(n[None, :] > n[:, None], -INF)
        return (torch.einsum("hij,jhd->ihd", sc.softmax(-1), vv[0].repeat_interleave(H // hkv, 1)) * do[0].double()).sum()

    xs = [t.double().requires_grad_() for t in (q, k, v)]
    want = torch.autograd.grad(loss(*xs), xs)
    for got, w in zip((dq, dk, dv), want):
        assert float((got.double() - w).norm() / w.norm()) <= tol
    for i, got in ((0, dq), (1, dk)):
        u = torch.randn(got.shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-5
        at = [t.detach().clone() for t in xs]
        at[i] = xs[i].detach() + h * u
        up = loss(*at)
        at[i] = xs[i].detach() - h * u
        diff = float((up - loss(*at)) / (2 * h))
        # (the differences' own error, h^2 of a third derivative, is far below)
        assert abs(float((got.double() * u).sum()) - diff) <= tol * float(got.double().norm()) * float(u.norm())


def test_a_captured_graph_and_another_stream():
    g = gen(8)
    q, k = rand(g, 300, 8, 128), rand(g, 300, 2, 128)
    cos, sin = ref.tables(600, 128, DEV)
    pos = torch.arange(300, device=DEV)
    out_q, out_k = torch.empty_like(q), torch.empty_like(k)
    run = lambda **kw: api.attn_rope(q, k, cos, sin, pos, out_q=out_q, out_k=out_k, **kw)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    pos.add_(123)
    q.copy_(rand(g, 300, 8, 128))
    graph.replay()
    torch.cuda.synchronize()
    want = api.attn_rope(q, k, cos, sin, pos)
    assert torch.equal(out_q, want[0]) and torch.equal(out_k, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.attn_rope(q, k, cos, sin, pos, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty_problems_and_refusals():
    cos, sin = ref.tables(8, 64, DEV)
    q = rand(gen(9), 8, 4, 64)
    a, b = api.attn_rope(q[:0], q[:0], cos, sin)
    assert a.shape == (0, 4, 64) and b.shape == (0, 4, 64)
    a, _ = api.attn_rope(q[:, :0], q, cos, sin)
    assert a.shape == (8, 0, 64)
    pos = torch.arange(8, device=DEV)
    bad = [
        (dict(q=q.float()), "bf16"), (dict(q=q.transpose(0, 1)), "contiguous"), (dict(k=q[:4]), "k must have"),
        (dict(cos=cos.double()), "float32"), (dict(sin=sin[:4]), "float32"), (dict(positions=pos.int()), "int64"),
        (dict(positions=pos[:4]), "positions"), (dict(positions=pos, pair_axis=(0,) * 31), "pair_axis"),
        (dict(positions=pos[None], pair_axis=(0, 1) * 16), "leading"), (dict(positions=pos[None], pair_axis=(0, 4) * 16), "axes"),
        (dict(pair_axis=(0,) * 32), "positions"), (dict(out_q=torch.empty_like(q)[:4]), "shapes"),
    ]
    for kw, match in bad:
        kw = dict(dict(q=q, k=q, cos=cos, sin=sin), **kw)
        with pytest.raises(ValueError, match=match):
            api.attn_rope(kw.pop("q"), kw.pop("k"), kw.pop("cos"), kw.pop("sin"), **kw)
    with pytest.raises(api.AttnError, match="shorter"):
        api.attn_rope(rand(gen(9), 9, 4, 64), None, cos, sin)
    with pytest.raises(api.AttnError, match="overlaps"):
        x = rand(gen(9), 9, 4, 64)
        api.attn_rope(x[:8], None, cos, sin, out_q=x[1:])
    with pytest.raises(api.AttnError, match="written"):
        api.attn_rope(q[:, :2], q[:, 2:], cos, sin, out_q=q[:, :2], out_k=q[:, :2])
