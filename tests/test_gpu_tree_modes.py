"""Trees of drafts in the modes of their own plans that the shapes of test_gpu_tree.py
leave out (tests/test_tree_plan_cpu.py derives which there are): few and short ones that
stream with more rows than chains do, 32 nodes to a path's last bit, ranges of prefix and
own tokens planned together, one range written without a join, one row tile and several.
Nodes stand in any order, some rows are none."""
import math

import pytest
import torch

from exact_attention_71_gb300 import api
from tests.test_gpu_paged import NAN, gen
from tests.test_gpu_tree import Tree, random_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"

MODES = [
    # lens, prefix, Nq, H, H_kv, d, page
    # streaming with 8 rows
    ([100], 300, 4, 4, 2, 64, 16),
    ([100], 300, 8, 1, 1, 128, 16),
    ([300], 100, 2, 8, 2, 256, 32),
    ([60, 3, 0], 0, 8, 2, 2, 256, 16),
    ([3000], 0, 7, 2, 2, 64, 16),
    # with 16, up to 16 or 32 rows
    ([40, 9], 60, 3, 10, 2, 64, 16),
    ([700], 900, 8, 4, 2, 256, 16),
    ([60, 16], 0, 16, 2, 2, 256, 16),
    # more rows, with and without a prefix, one range and several; 32 nodes
    ([60, 40, 32], 0, 32, 4, 2, 64, 16),
    ([100, 70], 40, 32, 16, 2, 64, 16),
    ([700, 300, 32], 0, 32, 8, 4, 64, 16),
    ([100, 33], 0, 32, 4, 1, 128, 32),
    ([96, 33], 0, 32, 4, 2, 128, 16),
    ([400, 330, 90], 500, 32, 4, 2, 128, 16),
    ([50, 41, 30], 0, 30, 3, 1, 256, 16),
    ([200, 150], 130, 32, 4, 2, 256, 16),
    # the prefix in tiles, own tokens streaming
    ([90, 60] * 20, 900, 12, 4, 2, 64, 16),
    # tiles, one and several, over the prefix and over own tokens
    ([300, 290], 700, 40, 2, 2, 64, 16),
    ([200, 77], 300, 40, 3, 3, 128, 16),
    ([300], 4000, 40, 2, 2, 256, 64),
    ([100, 0, 61], 0, 60, 2, 2, 64, 32),
    ([100, 90], 0, 80, 2, 1, 64, 16),
    ([300, 200], 0, 40, 3, 1, 128, 16),
    ([100, 90], 0, 80, 2, 1, 128, 16),
    ([50, 0, 41], 0, 40, 2, 2, 256, 16),
    ([48, 0, 41], 0, 40, 2, 2, 256, 16),
    ([44, 40], 0, 36, 8, 2, 256, 16),
]


def plan(shape):
    lens, prefix, Nq, H, hkv, d, ps = shape
    per = max(1, -(-max(lens + [1]) // ps)) + 1                # (pages of a row of Problem's table)
    return api.paged_tree_plan(len(lens), Nq, H, hkv, d, prefix, per, ps)


def shape_id(s):
    return "x".join(map(str, s[1:])) + "_" + str(len(s[0]))


def shuffled_parents(seed, B, Nq, width, none):
    """Random trees whose nodes stand in any order; about `none` of the rows are no nodes
    (what hung below them has no parent)."""
    g = gen(seed)
    p = random_parents(g, B, Nq, width).long()
    drop = torch.rand((B, Nq), generator=g, device=DEV) < none
    p = torch.where((p >= 0) & drop.gather(1, p.clamp(min=0)), torch.full_like(p, -1), p)
    to = torch.rand((B, Nq), generator=g, device=DEV).argsort(1)       # node i comes to stand at to[i]
    moved = torch.where(p >= 0, to.gather(1, p.clamp(min=0)), p)
    moved = torch.where(drop, torch.full_like(p, -3), moved)
    return torch.empty_like(p).scatter_(1, to, moved).to(torch.int32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", MODES, ids=shape_id)
def test_tree_attention_matches_the_plain_form(shape, fp8):
    B, Nq = len(shape[0]), shape[2]
    for seed, width in ((71, max(1, Nq // 4)), (72, 1)):              # a bush, chains (32 nodes deep)
        p = Tree(*shape, fp8=fp8, seed=seed, parents=shuffled_parents(seed, B, Nq, width, 0.15 if seed == 71 else 0.0))
        o, lse = p.run()
        p.check(o, lse)
        none = p.parents < -1
        assert bool((o[none] == 0).all()) and bool((lse.transpose(1, 2)[none] == -math.inf).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", MODES, ids=shape_id)
def test_a_value_that_is_not_finite_reaches_the_nodes_that_see_it_alone(shape, fp8):
    """One draft of every sequence, the last node with a child first: NaN in those that see
    it, the same bits in the others."""
    lens, _, Nq, H, hkv, d, ps = shape
    B = len(lens)
    p = Tree(*shape, fp8=fp8, seed=73, parents=shuffled_parents(73, B, Nq, 3, 0.1))
    o0, l0 = p.run()
    p.check(o0, l0)
    sees = torch.zeros((B, Nq), dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        nodes = [j for j in range(Nq) if int(p.parents[b, j]) > -2 and n - Nq + j >= 0]
        if not nodes:
            continue
        paths = p.rows(b)
        bad = max(nodes, key=lambda j: (sum(s is not None and j in s for s in paths) > 1, j))
        at = n - Nq + bad
        slot = torch.tensor([int(p.table[b, at // ps]) * ps + at % ps], device=DEV)
        v = p.v[b + 1][at:at + 1].clone()
        v[..., 3] = NAN
        api.attn_kv_write(p.k[b + 1][at:at + 1], v, slot, p.cache)
        sees[b] = torch.tensor([s is not None and bad in s for s in paths], device=DEV)
    assert bool(sees.any())
    o, l = p.run()
    assert api.device_status()[0] == 0
    l, l0 = l.transpose(1, 2), l0.transpose(1, 2)
    assert torch.equal(o[~sees], o0[~sees]) and torch.equal(l[~sees], l0[~sees])
    assert bool(torch.isnan(o[sees]).all()) and bool(torch.isnan(l[sees]).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d, B, Nq, G", [(64, 40, 12, 2), (128, 40, 12, 2), (256, 20, 12, 2)])
def test_rows_behind_a_prefix_whose_first_tiles_are_padding(d, B, Nq, G, fp8):
    """Row tiles of the prefix without a node anywhere: at the start, in between."""
    p = Tree([Nq + 5 * (b % 4) for b in range(B)], 700, Nq, 2 * G, 2, d, 16, fp8, seed=74, width=3)
    assert plan((p.lens, 700, Nq, 2 * G, 2, d, 16)).prefix_kernel == "tile"
    for gone in (slice(0, 8), slice(3, 9), slice(1, Nq)):
        p.parents = random_parents(gen(75), B, Nq, 2)
        p.parents[:, gone] = -2
        p.parents = torch.where((p.parents >= gone.start) & (p.parents < gone.stop), -1, p.parents).to(torch.int32)
        o, lse = p.run()
        p.check(o, lse)
        assert bool((o[:, gone] == 0).all()) and bool((lse[:, :, gone] == -math.inf).all())
