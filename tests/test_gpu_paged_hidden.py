"""What a query row of the paged attention sees and does not see, at its edges:
value rows that are not finite, and value scales far above the others."""
import pytest
import torch

from exact_attention_71_gb300 import api
from tests import paged_ref as ref
from tests.test_gpu_paged import DEV, INF, NAN, Problem

pytestmark = pytest.mark.gpu


def place(p, b, at):
    """(page, row) of token `at` of sequence b."""
    return int(p.table[b, at // p.ps]), at % p.ps


def write_value(p, b, at, value):
    """Token `at` of sequence b gets a value row with `value` in column 3."""
    page, row = place(p, b, at)
    y = p.v[b + 1][at:at + 1].clone()
    y[..., 3] = value
    api.attn_kv_write(p.k[b + 1][at:at + 1], y, torch.tensor([page * p.ps + row], device=DEV), p.cache)


# (lens, Nq, H, H_kv, d, tokens before the end) of both kernels: drafts and chunks, the
# key among the last ones.
NEAR = [
    ([70, 21], 4, 4, 2, 128, 1),
    ([70, 5], 5, 2, 2, 64, 2),
    ([300, 33], 3, 4, 1, 256, 2),
    ([170, 93], 80, 4, 2, 128, 5),
    ([170, 93], 80, 2, 2, 64, 5),
    ([170, 93], 80, 4, 2, 256, 1),
]
# The key lies among the last Nq - 1, but before the limit of every row of a CTA that
# sees it: some key tiles before it (or within one, of the streaming kernel's tiles of
# 16 rows).
FAR = [
    ([700, 600], 512, 8, 2, 128, 300),       # pairs of row tiles
    ([700, 640], 512, 2, 2, 64, 500),
    ([700, 640], 512, 4, 2, 256, 130),
    ([700, 640], 300, 2, 2, 128, 129),       # an odd number of row tiles
    ([300, 260], 100, 1, 1, 128, 60),        # one row tile
    ([300, 260], 16, 4, 2, 128, 11),         # streaming kernel, several row tiles
    ([90, 260], 16, 2, 1, 64, 12),
    ([300, 33], 16, 1, 1, 256, 9),
]


def shape_id(s):
    return f"{s[1]}x{s[2]}x{s[4]}_{s[5]}"


def check_row(p, back, before, change):
    """`change` makes the value row `back` tokens before each sequence's end not
    finite: the queries that see it are NaN, O and LSE, the others as before."""
    o0, l0 = before
    for b, n in enumerate(p.lens):
        change(b, n - back)
    o1, l1 = p.run()
    assert api.device_status()[0] == 0
    free = p.Nq - back                       # queries before the key
    assert torch.equal(o1[:, :free], o0[:, :free]) and torch.equal(l1[:, :, :free], l0[:, :, :free])
    assert bool(torch.isnan(o1[:, free:]).all()) and bool(torch.isnan(l1[:, :, free:]).all())


def check_code_or_scale(shape, what):
    lens, Nq, H, hkv, d, back = shape
    p = Problem(lens, 40, Nq, H, hkv, d, 32, True, seed=52)
    before = p.run()

    def change(b, at):
        page, row = place(p, b, at)
        if what == "code":
            p.cache.v[page, :, row, d - 2] = 0xff
        else:
            p.cache.v_scale[page, :, row] = NAN if what == "nan_scale" else INF

    check_row(p, back, before, change)


@pytest.mark.parametrize("what", ["code", "nan_scale", "inf_scale"])
@pytest.mark.parametrize("shape", NEAR, ids=shape_id)
def test_a_value_code_or_scale_that_is_not_finite(shape, what):
    check_code_or_scale(shape, what)


@pytest.mark.parametrize("what", ["code", "nan_scale", "inf_scale"])
@pytest.mark.parametrize("shape", FAR, ids=shape_id)
def test_the_same_far_before_the_limits_of_the_queries_that_see_it(shape, what):
    check_code_or_scale(shape, what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", NEAR + FAR, ids=shape_id)
def test_every_query_that_sees_a_value_row_that_is_not_finite_is_nan(shape, fp8):
    lens, Nq, H, hkv, d, back = shape
    p = Problem(lens, 40, Nq, H, hkv, d, 16, fp8, seed=51)
    before = p.run()
    check_row(p, back, before, lambda b, at: write_value(p, b, at, NAN if b == 0 else INF))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", FAR, ids=shape_id)
def test_a_query_that_is_not_finite_stays_alone(shape, fp8):
    """Its row of O says nothing about the values."""
    lens, Nq, H, hkv, d, back = shape
    p = Problem(lens, 40, Nq, H, hkv, d, 16, fp8, seed=55)
    o0, l0 = p.run()
    p.q[:, Nq - 2] = NAN
    o1, l1 = p.run()
    assert bool(torch.isnan(o1[:, Nq - 2]).all()) and bool(torch.isnan(l1[:, :, Nq - 2]).all())
    o1[:, Nq - 2] = o0[:, Nq - 2]
    l1[:, :, Nq - 2] = l0[:, :, Nq - 2]
    assert torch.equal(o1, o0) and torch.equal(l1, l0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", FAR, ids=shape_id)
def test_a_value_row_that_every_query_sees_stays_in_its_columns(shape, fp8):
    """The last key before the queries' own, and one of the prefix: LSE does not
    depend on the values; a bf16 infinity reaches its own column alone."""
    lens, Nq, H, hkv, d, _ = shape
    for where in ("own", "prefix"):
        p = Problem(lens, 40, Nq, H, hkv, d, 16, fp8, seed=53)
        o0, l0 = p.run()
        for b, n in enumerate(p.lens):
            if where == "own":
                if n > Nq:
                    write_value(p, b, n - Nq, INF)
            elif b == 0:
                slot = int(p.prefix_table[1]) * 16 + 3
                y = p.v[0][19:20].clone()
                y[..., 3] = INF
                api.attn_kv_write(p.k[0][19:20], y, torch.tensor([slot], device=DEV), p.cache)
        o1, l1 = p.run()
        assert torch.equal(l1, l0)
        if fp8:
            assert bool(torch.isnan(o1).all())          # the row's scale is NaN
        else:
            assert not bool(torch.isfinite(o1[..., 3]).any())
            for x, y in ((o1[..., :3], o0[..., :3]), (o1[..., 4:], o0[..., 4:])):
                assert torch.equal(x, y)


@pytest.mark.parametrize("exponent", [20, 60])
@pytest.mark.parametrize("shape", NEAR + FAR, ids=shape_id)
def test_a_large_value_scale_reaches_only_the_queries_that_see_it(shape, exponent):
    """e4m3: a row's values may be 2^20 or 2^60 times the others'.  Queries before it
    keep every bit; the others have it, and LSE is the same for all."""
    lens, Nq, H, hkv, d, back = shape
    p = Problem(lens, 40, Nq, H, hkv, d, 32, True, seed=54)
    o0, l0 = p.run()
    big = []
    for b, n in enumerate(p.lens):
        page, row = place(p, b, n - back)
        p.cache.v_scale[page, :, row] *= 2.0 ** exponent
        v = p.values("v", b)
        v[n - back] *= 2.0 ** exponent
        big.append(v)
    o1, l1 = p.run()
    assert api.device_status()[0] == 0
    free = Nq - back
    assert torch.equal(o1[:, :free], o0[:, :free]) and torch.equal(l1, l0)
    for b, n in enumerate(p.lens):
        k = torch.cat([p.values("k", -1), p.values("k", b)])
        v = torch.cat([p.values("v", -1), big[b]])
        q = p.q[b, free:].double()
        sees = [p.prefix + max(0, n - Nq + 1 + i) for i in range(free, Nq)]
        want, wl, spread, size = ref.attend(q, k, v, sees)
        to, _ = ref.tolerances(want, wl, spread, size, d)
        assert bool(((o1[b, free:].double() - want).abs() <= to).all()), b


def check_against_scaled_values(p, exponents, o, lse):
    """The plain form with the value rows of sequence b times 2^exponents[b]."""
    for b, n in enumerate(p.lens):
        k = torch.cat([p.values("k", -1), p.values("k", b)])
        v = torch.cat([p.values("v", -1), p.values("v", b) * torch.exp2(exponents[b].double())[:, None, None]])
        sees = [p.prefix + max(0, n - p.Nq + 1 + i) for i in range(p.Nq)]
        want, wl, spread, size = ref.attend(p.q[b].double(), k, v, sees)
        to, tl = ref.tolerances(want, wl, spread, size, p.d)
        for i in range(p.Nq):
            # weights or ratios of scales that fp16 rounds to a multiple of 2^-24, off
            # by 2^-25 of the largest that the query sees at most, for each of its keys
            if sees[i]:
                to[i] += sees[i] * 2.0 ** -25 * float(v[:sees[i]].abs().max())
        assert bool(((o[b].double() - want).abs() <= to).all()), b
        seen = torch.isfinite(wl)
        assert bool(((lse[b].double() - wl).abs()[seen] <= tl[seen]).all()), b


def check_random_scales(shape, back):
    lens, Nq, H, hkv, d, _ = shape
    p = Problem(lens, 40, Nq, H, hkv, d, 16, True, seed=56)
    g = torch.Generator(device=DEV).manual_seed(57)
    exponents = []
    for b, n in enumerate(lens):
        e = torch.zeros(n, device=DEV)
        tail = max(0, n - Nq - back)
        e[tail:] = torch.randint(-30, 61, (n - tail,), generator=g, device=DEV).float()
        for at in range(tail, n):
            page, row = place(p, b, at)
            p.cache.v_scale[page, :, row] *= 2.0 ** float(e[at])
        exponents.append(e)
    o, lse = p.run()
    assert api.device_status()[0] == 0
    check_against_scaled_values(p, exponents, o, lse)


@pytest.mark.parametrize("back", [-1, 3, 40])
@pytest.mark.parametrize("shape", NEAR + FAR + [([9, 3], 12, 2, 1, 128, 1), ([20, 1], 32, 1, 1, 64, 1), ([60, 130], 129, 2, 2, 128, 1)],
                         ids=shape_id)
def test_value_scales_of_the_last_tokens_from_2_to_the_minus_30_to_2_to_the_60(shape, back):
    """Each query against the plain form over the keys that it sees: from the second
    query's key on, from some keys before, and with sequences shorter than the
    queries."""
    check_random_scales(shape, back)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_value_row_that_is_not_finite_counts_however_small_its_weight_is(d, prefix, fp8):
    """One row tile, the keys in two halves: the second half's scores are 200 below the
    first's, so that its weights are 0 in binary32.  Its infinity still makes the
    queries that see it NaN."""
    Nq, n, back = 60, 500, 40
    p = Problem([n, n - 30], prefix, Nq, 1, 1, d, 16, fp8, seed=58)
    p.q[..., 0] = 40.0
    for b, ks in enumerate(p.k):
        ks[..., 0] = 0.0
        if b:
            ks[len(ks) // 2:, :, 0] = -5.0 * d ** 0.5
        t = p.prefix_table if b == 0 else p.table[b - 1]
        at = torch.arange(len(ks), device=DEV)
        if len(ks):
            api.attn_kv_write(ks, p.v[b], t.long()[at // 16] * 16 + at % 16, p.cache)
    before = p.run()
    assert bool(torch.isfinite(before[0]).all())
    check_row(p, back, before, lambda b, at: write_value(p, b, at, INF))
