"""The paged attention in the modes that the shapes of test_gpu_paged.py leave out
(tests/test_paged_plan_cpu.py derives which there are): one range written without
a join, by either kernel; 16-row streaming CTAs at head dim 256; several row tiles
of head dim 256 over own tokens in ranges, one of head dim 64 over a prefix."""
import math

import pytest
import torch

from exact_attention_71_gb300 import api
from tests.test_gpu_paged import INF, NAN, Problem
from tests.test_gpu_paged_hidden import check_row, write_value

pytestmark = pytest.mark.gpu

MODES = [
    # lens, prefix, Nq, H, H_kv, d, page
    # tile kernel, written without a join: two row tiles, one, an odd number of them
    ([100, 90], 0, 80, 2, 1, 64, 16),
    ([100, 0, 61], 0, 60, 2, 2, 64, 32),
    ([100, 90], 0, 80, 2, 1, 128, 16),
    ([100, 0, 61], 0, 60, 2, 2, 128, 32),
    ([110, 97], 0, 100, 3, 1, 128, 16),
    ([44, 33], 0, 80, 2, 1, 256, 16),
    ([40, 0, 17], 0, 20, 2, 2, 256, 16),
    # the same over several key tiles
    ([300] * 9 + [131], 0, 64, 32, 8, 128, 16),
    ([300] * 19 + [77], 0, 40, 8, 8, 128, 16),
    ([300] * 19 + [77], 0, 20, 8, 8, 256, 16),
    ([300] * 19 + [77], 0, 40, 8, 8, 64, 16),
    # streaming kernel, written without a join
    ([100, 3, 0], 0, 1, 2, 1, 256, 64),
    ([100, 90], 0, 12, 2, 2, 64, 16),
    ([100, 90], 0, 3, 16, 4, 128, 16),
    ([100, 3], 0, 12, 2, 2, 256, 64),
    # 16-row CTAs at d = 256, over the prefix and over own tokens, some and many ranges
    ([300], 100, 12, 2, 2, 256, 64),
    ([3000], 1500, 5, 6, 2, 256, 128),
    ([300, 90], 100, 12, 2, 2, 256, 64),
    # two row tiles of d = 256 over own tokens in ranges, one of d = 64 over a prefix
    ([200, 133], 0, 80, 2, 1, 256, 16),
    ([40, 90], 500, 20, 4, 2, 64, 16),
]


def plan(shape):
    lens, prefix, Nq, H, hkv, d, ps = shape
    per = max(1, -(-max(lens + [1]) // ps)) + 1                # (pages of a row of Problem's table)
    return api.paged_plan(len(lens), Nq, H, hkv, d, prefix, per, ps)


def shape_id(s):
    return "x".join(map(str, s[1:])) + "_" + str(len(s[0]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", MODES, ids=shape_id)
def test_attention_matches_the_plain_form(shape, fp8):
    p = Problem(*shape, fp8=fp8, seed=61)
    p.check(*p.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", MODES[:7] + MODES[11:16], ids=shape_id)
def test_without_the_causal_mask_every_own_key_is_seen(shape, fp8):
    p = Problem(*shape, fp8=fp8, seed=62)
    p.check(*p.run(causal=False), causal=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape, back", [
    (([260, 140] * 5, 0, 130, 32, 8, 128, 16), 60), (([260, 140] * 5, 0, 130, 32, 8, 64, 16), 100),
    (([100, 130] * 10, 0, 96, 16, 8, 256, 16), 70), (([90, 100], 0, 60, 4, 4, 128, 16), 20), (([60, 90], 0, 8, 4, 2, 256, 32), 5),
    (([60, 90], 0, 16, 4, 2, 64, 32), 12),
], ids=lambda x: str(x) if isinstance(x, int) else shape_id(x))
def test_rows_that_see_a_value_row_that_is_not_finite_are_written_as_nan(shape, back, fp8):
    assert plan(shape).direct
    p = Problem(*shape, fp8=fp8, seed=63)
    before = p.run()
    check_row(p, back, before, lambda b, at: write_value(p, b, at, NAN if b % 2 == 0 else -INF))
    assert api.device_status()[0] == 0


@pytest.mark.parametrize("shape", [MODES[2], MODES[4], MODES[11], MODES[15]], ids=shape_id)
def test_outputs_around_the_result_are_left_alone(shape):
    """o and lse inside larger buffers: nothing before or behind them is written."""
    p = Problem(*shape, fp8=True, seed=64)
    want = p.run()
    room = [torch.full((x.numel() + 256,), 7.0, dtype=x.dtype, device=x.device) for x in want]
    got = [r[128:-128].view(x.shape) for r, x in zip(room, want)]
    p.run(out=got[0], lse=got[1])
    for r, g, x in zip(room, got, want):
        assert torch.equal(g, x)
        assert bool((r[:128] == 7.0).all()) and bool((r[-128:] == 7.0).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix", [0, 16])
def test_more_sequences_than_a_grid_dimension_has(prefix, fp8):
    """70000 sequences of one token each (of its own: every result is that token's
    values, behind a prefix of another page: of the two)."""
    B, d = 70000, 64
    cache = api.kv_cache(B + 1, 16, 1, d, e4m3=fp8)
    g = torch.Generator(device="cuda").manual_seed(71)
    x = torch.randn((B, 1, d), generator=g, device="cuda").to(torch.bfloat16)
    api.attn_kv_write(x, x, torch.arange(B, device="cuda") * 16, cache)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    own = api.attn_kv_read(cache, table[:60000], lens[:60000], 1)[1][:, 0]
    if prefix:           # a page of zeros: 16 more keys with score 0 and value 0
        pages = torch.full((1,), B, dtype=torch.int32, device="cuda")
        q = torch.zeros((B, 1, 1, d), dtype=torch.bfloat16, device="cuda")
        o, lse = api.attn_fwd_paged(q, cache, table, lens, pages, prefix)
        want = own.double() / 17
        assert bool(((lse.double() - math.log(17.0)).abs() <= 2.0 ** -18).all())
    else:
        o, lse = api.attn_fwd_paged(x[:, None], cache, table, lens)
        want = own.double()
    assert api.device_status()[0] == 0
    # one weight of 1 (or 17 equal ones): values of the cache as they are, two
    # roundings to fp16 on the way at most and one to bf16; read back, one to bf16
    tol = 2 * 2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -20
    assert bool(((o[:60000, 0].double() - want).abs() <= tol * want.abs() + 1e-30).all())
    assert bool((o[60000:].float().abs().amax(-1) > 0).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kernel, B, N, Nq, sites", [("stream", 48, 8192, 1, (0xb1,)),
                                                     ("tile", 2, 2048, 90, tuple(range(0xa1, 0xac)))])
def test_a_wait_that_runs_out_is_reported_by_its_kernel(kernel, B, N, Nq, sites, fp8):
    """With a limit of one cycle the first hardware wait that ends without its copy (or
    product) gives up: the call is reported, by a site of the kernel that has all of
    its work, and the next one is right.  (Hardware waits last some microseconds: it
    takes a cache of a gigabyte for a copy of the streaming kernel to be that late.)"""
    H, hkv, d, ps = 32, 8, 128, 64
    p = api.paged_plan(B, Nq, H, hkv, d, 0, N // ps, ps)
    assert p.prefix_kernel is None and p.own_kernel == kernel
    cache = api.kv_cache(B * N // ps, ps, hkv, d, e4m3=fp8)
    g = torch.Generator(device="cuda").manual_seed(65)
    for t in cache[:2]:
        if fp8:
            t.random_(0, 0x70, generator=g)
        else:
            t.normal_(generator=g)
    q = torch.randn((B, Nq, H, d), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(B * N // ps, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    want = api.attn_fwd_paged(q, cache, table, lens)
    assert api.device_status()[0] == 0
    assert api.library().attn_set_wait_limit(1) == 0
    try:
        api.attn_fwd_paged(q, cache, table, lens)
        rc, site = api.device_status()
    finally:
        api.library().attn_set_wait_limit(0)
    assert rc == -4 and site in sites, (rc, hex(site))
    got = api.attn_fwd_paged(q, cache, table, lens)
    assert api.device_status()[0] == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_allocations_are_seen_by_modes_and_filled_where_torch_fills(monkeypatch):
    """The binding's quick way to allocate is taken only where nobody could tell."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.made = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            r = func(*args, **(kwargs or {}))
            if "empty" in str(func):
                self.made.append(tuple(r.shape))
            return r

    p = Problem([300, 77, 0], 900, 3, 8, 2, 128, 16, True, seed=66)
    want = p.run()
    with Seen() as mode:
        got = p.run()
    assert tuple(want[0].shape) in mode.made and tuple(want[1].shape) in mode.made and len(mode.made) == 3
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # (without the launch: what the outputs are allocated as)
    monkeypatch.setattr(api, "_launch", lambda *args: None)
    torch.use_deterministic_algorithms(True)
    try:
        o, lse = p.run()
        assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
    finally:
        torch.use_deterministic_algorithms(False)


@pytest.mark.parametrize("name", ["_raw_empty", "_raw_stream"])
def test_a_changed_signature_of_a_private_entry_costs_time_only(monkeypatch, name):
    p = Problem([300, 77, 0], 900, 3, 8, 2, 128, 16, True, seed=67)
    want = p.run()
    calls = []

    def changed(*args):
        calls.append(args)
        raise TypeError("one more argument")

    monkeypatch.setattr(api, name, changed)
    got = p.run()
    assert calls and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a mode's entry that changed: the public way
    monkeypatch.undo()
    monkeypatch.setattr(api, "_watchers", [changed])
    got = p.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    monkeypatch.setattr(api, "_watchers", [None])
    got = p.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
