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
