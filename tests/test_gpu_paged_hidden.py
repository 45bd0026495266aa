"""What a query row of the paged attention sees and does not see, at its edges:
value rows that are not finite."""
import pytest
import torch

from exact_attention_71_gb300 import api
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
