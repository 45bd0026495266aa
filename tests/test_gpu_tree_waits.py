"""Waits of the trees' kernels that run out are reported by the kernel that waited."""
import pytest
import torch

from exact_attention_71_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kernel, B, N, Nq, sites", [("stream", 48, 8192, 1, (0xb1,)),
                                                     ("tile", 2, 2048, 90, tuple(range(0xa1, 0xac)))])
def test_a_wait_that_runs_out_below_a_tree_is_reported_by_its_kernel(kernel, B, N, Nq, sites, fp8):
    """With a limit of one cycle the first hardware wait that ends without its copy (or
    product) gives up: the call is reported by a site of the kernel that has all of its
    work, and the next one is right.  (Hardware waits last some microseconds: it takes a
    cache of a gigabyte for a copy of the streaming kernel to be that late, and few query
    rows: with 16 an e4m3 cache's copies are ahead of the products.)"""
    H, hkv, d, ps = 32, 8, 128, 64
    p = api.paged_tree_plan(B, Nq, H, hkv, d, 0, N // ps, ps)
    assert p.prefix_kernel is None and p.own_kernel == kernel
    cache = api.kv_cache(B * N // ps, ps, hkv, d, e4m3=fp8)
    g = torch.Generator(device=DEV).manual_seed(65)
    for t in cache[:2]:
        if fp8:
            t.random_(0, 0x70, generator=g)
        else:
            t.normal_(generator=g)
    q = torch.randn((B, Nq, H, d), generator=g, device=DEV).to(torch.bfloat16)
    table = torch.arange(B * N // ps, dtype=torch.int32, device=DEV).view(B, -1)
    lens = torch.full((B,), N, dtype=torch.int32, device=DEV)
    parents = torch.arange(Nq, dtype=torch.int32, device=DEV) // 2 - 1
    want = api.attn_fwd_paged_tree(q, cache, table, lens, parents)
    assert api.device_status()[0] == 0
    assert api.library().attn_set_wait_limit(1) == 0
    try:
        api.attn_fwd_paged_tree(q, cache, table, lens, parents)
        rc, site = api.device_status()
    finally:
        api.library().attn_set_wait_limit(0)
    assert rc == -4 and site in sites, (rc, hex(site))
    got = api.attn_fwd_paged_tree(q, cache, table, lens, parents)
    assert api.device_status()[0] == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
