"""A speculative decoding step over the paged cache: appending with the rotation,
attention of a tree of drafts, accepting a path; against 64-bit forms."""
import math

import pytest
import torch

from exact_attention_71_gb300 import api
from tests import paged_ref, rope_ref as ref
from tests.test_gpu_paged import INF, NAN, Problem, cache_rows, code_values, filled_cache, gen, rand
from tests.test_gpu_rope_rows import sections

pytestmark = pytest.mark.gpu
DEV = "cuda"


def random_parents(g, B, Nq, width):
    back = 1 + (torch.rand((B, Nq), generator=g, device=DEV) * width).long().clamp(max=width - 1)
    return (torch.arange(Nq, device=DEV) - back).clamp(min=-1).to(torch.int32)


class Tree(Problem):
    """A Problem whose last Nq own tokens are a tree's nodes."""

    def __init__(self, *args, width=3, parents=None, **kw):
        super().__init__(*args, **kw)
        B = len(self.lens)
        self.parents = random_parents(gen(77), B, self.Nq, width) if parents is None else parents

    def run(self, **kw):
        return api.attn_fwd_paged_tree(self.q, self.cache, self.table, self.seq_lens, self.parents, self.prefix_table,
                                       self.prefix, **kw)

    def rows(self, b):
        p = self.parents if self.parents.dim() == 1 else self.parents[b]
        return ref.paths(p.tolist())

    def check(self, o, lse, scale=None, status=0):
        assert api.device_status()[0] == status
        for b, n in enumerate(self.lens):
            k = torch.cat([self.values("k", -1), self.values("k", b)])
            v = torch.cat([self.values("v", -1), self.values("v", b)])
            mask = torch.zeros((self.Nq, len(k)), dtype=torch.bool)
            for i, seen in enumerate(self.rows(b)):
                if seen is None:
                    continue
                mask[i, :self.prefix + max(0, n - self.Nq)] = True
                for j in seen:
                    if n - self.Nq + j >= 0:
                        mask[i, self.prefix + n - self.Nq + j] = True
            want, wl, spread, size = ref.attend(self.q[b].double(), k, v, mask.to(DEV), scale)
            to, tl = paged_ref.tolerances(want, wl, spread, size, self.d)
            err = (o[b].double() - want).abs()
            within = bool((err <= to).all())
            assert within, (b, float((err - to).max()), float(err.max()))
            empty = torch.isinf(wl)
            assert torch.equal(torch.isinf(lse[b]) & (lse[b] < 0), empty)
            dl = (lse[b].double() - wl).abs()[~empty]
            within = bool((dl <= tl[~empty]).all())
            assert within, (b, float(dl.max()))


# lens, prefix, Nq, H, H_kv, d, page, width: both kernels over the tokens before the
# drafts, one, two and four warps a tile, tiles of several nodes and of one node's heads,
# pages that end inside the drafts, drafts that fill whole pages, chains and bushes.
SHAPES = [
    ([1], 0, 1, 1, 1, 64, 16, 1),                    # nothing but the node itself
    ([0, 1, 2, 17], 0, 1, 4, 2, 128, 16, 1),         # single tokens; an empty sequence
    ([5, 9, 40], 0, 5, 4, 4, 64, 16, 2),
    ([8, 300], 130, 8, 8, 2, 128, 32, 3),
    ([30, 21, 100, 0], 47, 21, 6, 3, 128, 16, 4),
    ([3, 70], 60, 7, 4, 2, 64, 16, 3),               # a sequence shorter than the tree
    ([64, 200], 0, 64, 8, 2, 128, 64, 12),
    ([130, 257], 33, 65, 4, 1, 256, 32, 20),
    ([333] * 3, 0, 100, 2, 2, 64, 16, 1),            # a chain of 100
    ([700], 1000, 16, 32, 1, 128, 128, 5),           # 32 heads a node: two tiles
    ([5000], 0, 13, 4, 1, 128, 16, 4),               # many ranges
    ([9000, 10], 0, 6, 2, 1, 64, 16, 3),
    ([600, 513], 300, 512, 1, 1, 64, 64, 60),        # the largest tree
    ([100] * 40, 2000, 4, 4, 2, 128, 16, 2),         # many rows behind the prefix
    ([60, 45], 4100, 33, 3, 1, 256, 256, 8),
    ([20000], 0, 2, 1, 1, 256, 64, 1),
    ([3000, 2900, 40], 0, 24, 16, 2, 128, 64, 4),    # up to 32 nodes in the tile kernel
    ([1500, 33], 3000, 32, 8, 1, 64, 32, 5),
    ([900, 800], 100, 20, 8, 2, 256, 32, 3),
    ([100, 70, 300], 40, 32, 16, 2, 64, 16, 6),      # and many rows of few, short ones, streaming
    ([41, 64], 300, 16, 24, 2, 256, 16, 3),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])) + "_" + str(len(s[0])))
def test_tree_attention_matches_the_plain_form(shape, fp8):
    p = Tree(*shape[:-1], fp8=fp8, seed=7, width=shape[-1])
    p.check(*p.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_one_tree_for_all_sequences_in_any_order_of_nodes(fp8):
    """Parents behind their children, several roots, rows that are no nodes."""
    parents = torch.tensor([3, -1, 0, -1, -2, 1, 5, -2, 2], dtype=torch.int32, device=DEV)
    p = Tree([90, 9, 41], 20, 9, 8, 2, 128, 16, fp8, seed=8, parents=parents)
    o, lse = p.run()
    p.check(o, lse)
    assert bool((o[:, [4, 7]] == 0).all()) and bool((lse[:, :, [4, 7]] == -math.inf).all())
    p.parents = parents.repeat(3, 1)
    o2, l2 = p.run()
    assert torch.equal(o, o2) and torch.equal(lse, l2)


# lens, prefix, Nq, H, H_kv, d, page; the plan: every way in which a row that is no node
# leaves the kernels (written at once, or told to either form of the join).
EMPTIES = [
    ([5 + b % 3 for b in range(300)], 0, 4, 8, 2, 64, 16, ("stream", True)),
    ([60 + b % 9 for b in range(70)], 0, 7, 16, 4, 64, 16, ("stream", True)),
    ([150 + b % 5 for b in range(160)], 0, 5, 8, 2, 128, 16, ("stream", True)),
    ([60 + b % 5 for b in range(160)], 0, 40, 2, 2, 128, 16, ("tile", True)),
    ([290 + b % 5 for b in range(160)], 0, 40, 2, 2, 128, 16, ("tile", True)),
    ([90, 41], 70, 4, 8, 2, 128, 16, ("stream", False)),
    ([9000, 70], 0, 6, 4, 1, 64, 16, ("stream", False)),               # many ranges
    ([5000, 300], 200, 40, 4, 1, 128, 64, ("tile", False)),
    ([700], 90, 130, 1, 1, 256, 64, ("tile", False)),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", EMPTIES, ids=lambda c: "x".join(map(str, c[1:])) + "_" + str(len(c[0])))
def test_rows_that_are_no_nodes_are_empty_in_every_mode(case, fp8):
    *shape, plan = case
    lens, _, Nq = shape[:3]
    parents = random_parents(gen(5), len(lens), Nq, 3)
    parents[:, Nq - Nq // 3:] = -2
    parents[-1] = -2                                   # a whole sequence without a tree
    p = Tree(*shape, fp8=fp8, seed=21, parents=parents)
    got = api.paged_plan(len(lens), Nq, shape[3], shape[4], shape[5], shape[1], p.table.shape[1], shape[6])
    assert (got.own_kernel, got.direct) == plan
    o, lse = p.run()
    p.check(o, lse)
    none = parents < -1
    assert bool((o[none] == 0).all()) and bool((lse.transpose(1, 2)[none] == -math.inf).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [2, 33, 64])
def test_many_sequences_of_any_lengths(B, fp8):
    """More CTAs than multiprocessors: long sequences are taken first, each of them once."""
    lens = [(0, 700, 41, 333, 700, 699, 5, 128)[(5 * b + b // 8) % 8] for b in range(B)]
    H = 128 if B == 2 else 8
    p = Tree(lens, 0, 40, H, H, 64, 16, fp8, seed=21, width=6)
    assert api.paged_plan(B, 40, H, H, 64, 0, p.table.shape[1], 16).own_kernel == "tile"
    p.check(*p.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B, Nq, H, hkv, prefix", [(3, 5, 8, 2, 200), (3, 5, 8, 2, 9000), (40, 20, 8, 2, 700), (2, 70, 8, 2, 90),
                                                   (1, 33, 64, 1, 40)])
def test_empty_sequences_behind_a_prefix(B, Nq, H, hkv, prefix, fp8):
    """No own tokens: nodes see the prefix, other rows nothing; also with a table of no columns."""
    p = Tree([0] * B, prefix, Nq, H, hkv, 128, 16, fp8, seed=23, width=3)
    p.parents[:, Nq - Nq // 4:] = -2
    p.parents[B // 2, 0] = -2 if B > 1 else -1
    p.parents[B // 2, 1:] = torch.where(p.parents[B // 2, 1:] == -2, -2, -1).int()
    o, lse = p.run()
    p.check(o, lse)
    p.table = p.table[:, :0]
    o2, l2 = p.run()
    p.check(o2, l2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d, B, Nq, G", [(64, 20, 16, 4), (128, 37, 9, 2), (256, 3, 40, 5), (128, 130, 4, 1)])
def test_padded_trees_behind_a_prefix(d, B, Nq, G, fp8):
    """Tiles of the prefix's rows that are all padding are left out, also where every row is."""
    p = Tree([Nq + 3 * (b % 7) for b in range(B)], 700, Nq, 2 * G, 2, d, 16, fp8, seed=22, width=3)
    for b in range(B):
        p.parents[b, max(1, Nq - Nq // 3 - b % 3):] = -2
    p.parents[B // 2] = -2                                  # a slot without a tree
    p.parents[0, Nq - 1] = 0                                # one of the last nodes is there
    p.check(*p.run())
    p.parents[:] = -2
    o, lse = p.run()
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 256])
def test_the_largest_tree_and_a_value_that_is_not_finite_in_each_of_its_tiles(d, fp8):
    """512 nodes that begin inside a tile of keys; bad values 64 keys apart: each makes the
    nodes NaN that see it, and no other."""
    Nq, n = 512, 512 + 77
    p = Tree([n], 0, Nq, 1, 1, d, 32, fp8, seed=22, width=40)
    p.check(*p.run())
    o0, l0 = p.run()
    paths = p.rows(0)
    seen_by = lambda node: torch.tensor([node in s for s in paths], device=DEV)
    for node in range(13, Nq, 64):
        at = n - Nq + node
        slot = torch.tensor([int(p.table[0, at // 32]) * 32 + at % 32], device=DEV)
        v = p.v[1][at:at + 1].clone()
        v[..., 1] = NAN
        api.attn_kv_write(p.k[1][at:at + 1], v, slot, p.cache)
        o, l = p.run()
        sees = seen_by(node)
        assert bool(torch.isnan(o[0][sees]).all()) and torch.equal(o[0][~sees], o0[0][~sees])
        assert bool(torch.isnan(l[0, 0][sees]).all()) and torch.equal(l[0, 0][~sees], l0[0, 0][~sees])
        api.attn_kv_write(p.k[1][at:at + 1], p.v[1][at:at + 1], slot, p.cache)
    assert api.device_status()[0] == 0


def test_bad_parents_of_larger_trees():
    """The tile kernel's walk: out of range, circles, children of rows that are no nodes."""
    parents = torch.arange(-1, 79, dtype=torch.int32, device=DEV)
    for i, to in ((10, 200), (30, 40), (50, 50), (60, -2), (70, 1 << 30)):
        parents[i] = to
    for fp8 in (False, True):
        p = Tree([200, 81], 50, 80, 2, 1, 128, 16, fp8, seed=23, parents=parents)
        p.check(*p.run(), status=-5)
        p.run()
        assert api.device_status() == (-5, 0x105)


@pytest.mark.parametrize("case", [([168], 0, 40, 1, 1, 128, 16), ([168, 128 + 33], 0, 33, 4, 2, 64, 32), ([192], 0, 64, 1, 1, 256, 16),
                                  ([12, 9], 30, 8, 4, 2, 128, 16), ([40], 0, 32, 1, 1, 64, 16)])
def test_ranges_of_nodes_alone_with_scales_of_any_size(case):
    """A stream, a range or a warp that begins with nodes has no key that all rows see."""
    p = Tree(*case, fp8=True, seed=35, width=3)
    g = gen(36)
    for b, vs in enumerate(p.v):
        if b == 0:
            continue
        nodes = vs[-p.Nq:]
        nodes *= torch.exp2(torch.randint(-20, 21, (len(nodes), 1, 1), generator=g, device=DEV).float()).to(torch.bfloat16)
        nodes[::7] = 0.0
        i = torch.arange(len(vs), device=DEV)
        api.attn_kv_write(p.k[b], vs, p.table[b - 1].long()[i // p.ps] * p.ps + i % p.ps, p.cache)
    p.check(*p.run())


def test_a_chain_is_the_causal_mask():
    """The same tokens through attn_fwd_paged: each is within its own rounding of the
    same values (bf16 weights on one side, results in bf16 on both)."""
    for fp8 in (False, True):
        chain = torch.arange(-1, 11, dtype=torch.int32, device=DEV)
        p = Tree([300, 12, 77], 50, 12, 8, 2, 128, 16, fp8, seed=9, parents=chain)
        o, lse = p.run()
        c, cl = api.attn_fwd_paged(p.q, p.cache, p.table, p.seq_lens, p.prefix_table, p.prefix)
        assert float((o.float() - c.float()).abs().max()) <= 4 * 2.0 ** -8 * float(c.float().abs().max().clamp(min=1))
        assert float((lse - cl).abs().max()) <= 1e-4


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_parents_are_reported_and_make_their_node_none(fp8):
    for bad, none in (([-1, 0, 7, 2], [2, 3]), ([-1, 2, 1, 1], [1, 2, 3]), ([0, 0, 1, -1], [0, 1, 2]),
                      ([-1, -2, 1, 0], [1, 2]), ([1 << 30, -1, 1, 0], [0, 3]), ([-1, 0, 2, 1], [2])):
        p = Tree([40, 4], 20, 4, 4, 2, 64, 16, fp8, seed=10, parents=torch.tensor(bad, dtype=torch.int32, device=DEV))
        o, lse = p.run()
        p.check(o, lse, status=-5)
        assert bool((o[:, none] == 0).all()) and bool((lse[:, :, none] == -math.inf).all())
        p.run()
        assert api.device_status() == (-5, 0x105)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,Nq,G", [(64, 6, 1), (128, 20, 2), (256, 40, 2)])
def test_what_a_node_does_not_see_cannot_reach_it(d, Nq, G, fp8):
    """A draft's value row with a NaN or an infinity, then its key row, then its scale:
    the nodes that see it become NaN, the others keep their bits."""
    p = Tree([Nq + 61, Nq + 5], 30, Nq, 2 * G, 2, d, 16, fp8, seed=11, width=4)
    o0, l0 = p.run()
    p.check(o0, l0)
    bad = Nq // 2
    sees = torch.tensor([[s is not None and bad in s for s in p.rows(b)] for b in range(2)], device=DEV)
    assert bool(sees.any()) and not bool(sees.all())

    def same_elsewhere(o, l):
        assert torch.equal(o[~sees], o0[~sees]) and torch.equal(l.transpose(1, 2)[~sees], l0.transpose(1, 2)[~sees])
        assert bool(torch.isnan(o[sees]).all()) and bool(torch.isnan(l.transpose(1, 2)[sees]).all())
        assert api.device_status()[0] == 0

    def put(b, k, v):
        at = p.lens[b] - Nq + bad
        slot = torch.tensor([int(p.table[b, at // 16]) * 16 + at % 16], device=DEV)
        api.attn_kv_write(k, v, slot, p.cache)
        return int(slot)

    rows = [(p.k[b + 1][p.lens[b] - Nq + bad][None], p.v[b + 1][p.lens[b] - Nq + bad][None]) for b in range(2)]
    for b, value in ((0, NAN), (1, -INF)):
        v = rows[b][1].clone()
        v[..., d - 3] = value
        put(b, rows[b][0], v)
    same_elsewhere(*p.run())
    for b in range(2):
        put(b, torch.full_like(rows[b][0], NAN), rows[b][1])
    same_elsewhere(*p.run())
    if fp8:
        for b, value in ((0, INF), (1, NAN)):
            slot = put(b, *rows[b])
            p.cache.v_scale[slot // 16, :, slot % 16] = value
        same_elsewhere(*p.run())
        for b in range(2):                             # a NaN code among good ones
            slot = put(b, *rows[b])
            p.cache.v[slot // 16, :, slot % 16, 5] = 0xff if b else 0x7f
        same_elsewhere(*p.run())
    # finite, but far above the others: the rows that do not see it keep their bits too
    for b in range(2):
        v = rows[b][1] * (2.0 ** 60)
        put(b, rows[b][0], v)
        p.v[b + 1][p.lens[b] - Nq + bad] = v[0]
    o, l = p.run()
    assert torch.equal(o[~sees], o0[~sees]) and torch.equal(l, l0)
    p.check(o, l)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_of_drafts_outside_the_cache_are_reported_and_hidden(fp8):
    """Of drafts that no node sees (the results are the same), then of the nodes'."""
    parents = torch.tensor([-1, 0, 1, -2, -2, -2] + [-2] * 14, dtype=torch.int32, device=DEV)
    p = Tree([52], 0, 20, 4, 2, 128, 16, fp8, seed=12, parents=parents)          # drafts: tokens 32 to 51
    p.check(*p.run())
    p.table[0, 3] = -5                                 # tokens 48 to 51, no nodes
    o, lse = p.run()
    p.check(o, lse, status=-5)
    p.table[0, 2] = p.cache.k.shape[0]                 # the nodes' page
    o2, l2 = p.run()
    assert api.device_status() == (-5, 0x102)
    p.lens, p.Nq = [32], 20
    context = torch.ones((20, 32), dtype=torch.bool, device=DEV)
    context[3:] = False
    want, wl, spread, size = ref.attend(p.q[0].double(), p.values("k", 0)[:32], p.values("v", 0)[:32], context)
    to, tl = paged_ref.tolerances(want, wl, spread, size, 128)
    assert bool(((o2[0].double() - want).abs() <= to).all()) and bool(((l2[0].double() - wl).abs()[:, :3] <= tl[:, :3]).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_extreme_scores(fp8):
    """Scores of -800 in the context and around 0 in the drafts and the other way
    round, and scores that all lie far below 0."""
    for kind in range(3):
        p = Tree([200, 90], 100, 20, 4, 2, 64, 16, fp8, seed=13, width=4)
        p.q[..., 0] = 40.0
        for b, ks in enumerate(p.k):
            n = len(ks)
            ks[..., 0] = (-160.0, 0.0, -160.0)[kind]
            if b > 0:
                ks[n - 20:, :, 0] = (0.0, -160.0, -160.0)[kind]
            t = p.prefix_table if b == 0 else p.table[b - 1]
            i = torch.arange(n, device=DEV)
            api.attn_kv_write(ks, p.v[b], t.long()[i // 16] * 16 + i % 16, p.cache)
        p.check(*p.run())


def test_value_scales_that_differ_by_orders_of_magnitude():
    p = Tree([400, 90], 700, 40, 4, 2, 128, 16, True, seed=33, width=5)
    g = gen(34)
    for b, vs in enumerate(p.v):
        vs *= torch.exp2(torch.randint(-12, 13, (len(vs), 1, 1), generator=g, device=DEV).float()).to(torch.bfloat16)
        t = p.prefix_table if b == 0 else p.table[b - 1]
        i = torch.arange(len(vs), device=DEV)
        api.attn_kv_write(p.k[b], vs, t.long()[i // 16] * 16 + i % 16, p.cache)
    p.check(*p.run())


def test_tree_repeats_streams_given_buffers_and_two_calls_at_once():
    p = Tree([300, 200, 100, 40], 700, 9, 8, 2, 128, 16, True, seed=41)
    r = Tree([600, 64], 300, 64, 8, 2, 128, 16, False, seed=42, width=9)
    want = [p.run(), r.run()]
    p.check(*want[0])
    r.check(*want[1])
    need = api.paged_tree_workspace_bytes(4, 9, 8, 2, 128, 700, p.table.shape[1], 16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(p.q), torch.empty_like(want[0][1])
    got = p.run(out=out, lse=lse, workspace=ws)
    assert got[0] is out and torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
    with pytest.raises(api.AttnError, match="smaller"):
        p.run(workspace=ws[:need - 256])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [x.run(stream=s) for x, s in zip((p, r), streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_waits_that_run_out_below_a_tree_are_reported():
    lib = api.library()
    for Nq in (4, 40):
        p = Tree([2000, 1500], 2000, Nq, 8, 2, 128, 64, True, seed=44)
        want = p.run()
        torch.cuda.synchronize()
        assert lib.attn_set_wait_limit(1) == 0
        try:
            p.run()
            rc, _ = api.device_status()
        finally:
            lib.attn_set_wait_limit(0)
        assert rc in (0, -4)
        got = p.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and api.device_status()[0] == 0


# ------------------------------------------------------------------ append

def appended(case, seed, pad=9, fp8=True):
    T, H, hkv, d, rot, axes, mixed, il, ps = case
    g = gen(seed)
    x = rand(g, T, H + 2 * hkv, d)                                    # columns of a projection
    pages = T // ps + 3
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T]
    slots[::pad] = -1 - torch.arange(len(slots[::pad]), device=DEV)
    cos, sin = ref.tables(3001, rot, DEV)
    pos = torch.randint(0, 3001, (axes, T), generator=g, device=DEV)
    pos[:, ::pad] = -7                                                # (not looked at)
    return x[:, :H], x[:, H:H + hkv], x[:, H + hkv:], slots, cos, sin, pos, filled_cache(pages, ps, hkv, d, fp8)


APPENDS = [
    (1, 1, 1, 64, 64, 1, False, False, 16), (2, 4, 4, 128, 128, 1, False, True, 16), (32, 8, 2, 128, 128, 1, False, False, 64),
    (203, 3, 3, 64, 32, 2, False, True, 16), (131, 6, 1, 256, 256, 3, True, False, 128), (77, 5, 5, 128, 96, 3, False, False, 32),
    (5000, 9, 3, 128, 128, 3, False, False, 16), (4001, 7, 5, 64, 48, 1, False, True, 256), (3001, 4, 3, 256, 64, 2, True, False, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "x".join(map(str, c)))
def test_append_turns_and_writes(case, fp8):
    T, H, hkv, d, rot, axes, mixed, il, ps = case
    q, k, v, slots, cos, sin, pos, cache = appended(case, 3, fp8=fp8, pad=9 if T > 2 else 5)
    pair_axis = sections(rot // 2, axes, mixed)
    before = [None if t is None else t.clone() for t in cache]
    got = api.attn_kv_append(q, k, v, pos if axes > 1 else pos[0], slots, cache, cos, sin, pair_axis if axes > 1 else None, il)
    assert api.device_status()[0] == 0
    keep = slots >= 0
    c, s = ref.gather(cos, sin, pos[:, keep], pair_axis)
    want, size = ref.turn(q[keep], c, s, rot, il)
    assert bool(((got[keep].double() - want).abs() <= ref.rounding(want, size)).all())
    assert bool((got[~keep] == 0).all())
    page, row = slots[keep] // ps, slots[keep] % ps
    turned, _ = ref.turn(k[keep], c, s, rot, il, torch.float32)
    mask = torch.ones((cache.k.shape[0], ps), dtype=torch.bool, device=DEV)
    mask[page, row] = False
    mask = mask[:, None, :].expand(-1, hkv, ps)
    for n, x, y0, s0 in (("k", turned, before[0], before[2]), ("v", v[keep].float(), before[1], before[3])):
        y = getattr(cache, n)
        if fp8:
            codes, scale = ref.quantise(x)
            assert torch.equal(code_values(y)[page, :, row], codes)
            assert torch.equal(getattr(cache, n + "_scale")[page, :, row], scale)
            assert bool(torch.isnan(getattr(cache, n + "_scale")[mask]).all())
        else:
            assert torch.equal(y[page, :, row], x.to(torch.bfloat16))
        assert torch.equal(y[mask].view(torch.uint8), y0[mask].view(torch.uint8))


@pytest.mark.parametrize("T", [12, 5000])
def test_append_of_extreme_rows(T):
    """Zeros, the smallest and the largest numbers, infinities and NaN."""
    case = (T, 2, 2, 128, 128, 1, False, False, 16)
    q, k, v, slots, cos, sin, pos, cache = appended(case, 4, pad=T + 1)
    slots[0], pos[:, 0] = cache.k.shape[0] * 16 - 1, 5
    slots[1:] = torch.arange(T - 1, device=DEV)
    k, v = k.contiguous(), v.contiguous()
    k[0] = v[0] = 0.0
    k[1] = v[1] = torch.tensor(9.2e-41).to(torch.bfloat16)
    k[2] = k[2] * 1e-38
    k[3] = torch.finfo(torch.bfloat16).max / 2
    k[4] = k[4] * 1e30
    k[5, 0, 7] = INF
    k[6, 1, 70] = NAN
    api.attn_kv_append(None, k, v, pos[0], slots, cache, cos, sin)
    assert api.device_status()[0] == 0
    c, s = ref.gather(cos, sin, pos, (0,) * 64)
    turned, _ = ref.turn(k, c, s, 128, False, torch.float32)
    page, row = slots // 16, slots % 16
    scale = cache.k_scale[page, :, row]
    bad = torch.zeros((T, 2), dtype=torch.bool, device=DEV)
    bad[5, 0] = bad[6, 1] = True
    assert torch.equal(torch.isnan(scale), bad)
    codes, want = ref.quantise(torch.where(bad[..., None], 0.0, turned))
    assert torch.equal(scale[~bad], want[~bad])
    assert torch.equal(code_values(cache.k)[page, :, row][~bad], codes[~bad])


def test_append_refuses_slots_and_positions_out_of_range():
    for what in ("slot", "position"):
        for fp8 in (False, True):
            case = (40, 3, 2, 64, 64, 2, False, False, 16)
            q, k, v, slots, cos, sin, pos, cache = appended(case, 5, fp8=fp8)
            pair_axis = sections(32, 2, False)
            pos[:, ::9] = 0
            if what == "slot":
                slots[10], slots[11] = cache.k.shape[0] * 16, 1 << 50
            else:
                pos[1, 10], pos[0, 11] = 3001, -1
            same = slots.clone()
            same[10] = same[11] = -1
            other = filled_cache(cache.k.shape[0], 16, 2, 64, fp8)
            want = api.attn_kv_append(q, k, v, pos, same, other, cos, sin, pair_axis)
            assert api.device_status()[0] == 0
            got = api.attn_kv_append(q, k, v, pos, slots, cache, cos, sin, pair_axis)
            assert api.device_status() == (-5, 0x101 if what == "slot" else 0x104)
            assert torch.equal(got, want) and bool((got[10:12] == 0).all())
            for a, b in zip(cache, other):
                assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_in_place_and_binding_refusals():
    case = (50, 4, 2, 128, 128, 1, False, False, 16)
    q, k, v, slots, cos, sin, pos, cache = appended(case, 6)
    want = api.attn_kv_append(q, k, v, pos[0], slots, cache, cos, sin)
    saved = [t.clone() for t in cache]
    assert api.attn_kv_append(None, k, v, pos[0], slots, cache, cos, sin) is None
    kk, vv = k.clone(), v.clone()
    got = api.attn_kv_append(q, k, v, pos[0], slots, cache, cos, sin, out_q=q)
    assert got is q and torch.equal(q, want) and torch.equal(k, kk) and torch.equal(v, vv)
    for a, b in zip(cache, saved):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    args = dict(q=q, k=k, v=v, positions=pos[0], slots=slots)
    for change, match in ((dict(k=k[:, :1]), "k and v"), (dict(v=v[:4]), "k and v"), (dict(q=q[:4]), "q must"),
                          (dict(positions=pos), "positions"), (dict(positions=pos[0].int()), "positions"),
                          (dict(slots=slots.int()), "slots"), (dict(q=None, out_q=q), "without q"),
                          (dict(pair_axis=(0,) * 3), "pair_axis"), (dict(out_q=q[:, :2]), "shape")):
        kw = dict(args, **change)
        with pytest.raises(ValueError, match=match):
            api.attn_kv_append(kw.pop("q"), kw.pop("k"), kw.pop("v"), kw.pop("positions"), kw.pop("slots"), cache, cos, sin, **kw)
    with pytest.raises(api.AttnError, match="new keys"):
        x = rand(gen(1), 50, 6, 128)
        api.attn_kv_append(x[:, :2], x[:, 2:4], x[:, 4:], pos[0], slots, cache, cos, sin, out_q=x[:, 3:5])
    empty = api.attn_kv_append(q[:0], k[:0], v[:0], pos[0, :0], slots[:0], cache, cos, sin)
    assert empty.shape == (0, 4, 128)


def test_append_beyond_32_bit_offsets():
    ps, hkv, d = 256, 8, 256
    pages = (1 << 32) // (ps * hkv * d) + 2
    cache = api.kv_cache(pages, ps, hkv, d)
    g = gen(31)
    x = rand(g, 3, 3 * hkv, d)
    cos, sin = ref.tables(3, d, DEV)
    pos = torch.arange(3, device=DEV)
    slots = torch.tensor([pages * ps - 1, (pages - 1) * ps, 7], device=DEV)
    low = api.kv_cache(2, ps, hkv, d)
    api.attn_kv_append(x[:, :hkv], x[:, hkv:2 * hkv], x[:, 2 * hkv:], pos, slots, cache, cos, sin)
    api.attn_kv_append(x[:, :hkv], x[:, hkv:2 * hkv], x[:, 2 * hkv:], pos, torch.tensor([511, 256, 7], device=DEV), low, cos, sin)
    for a, b in zip(cache, low):
        assert torch.equal(a[-1], b[1]) and torch.equal(a[0], b[0])


# ------------------------------------------------------------------ accept

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,ps,hkv,Nq,M", [(64, 16, 3, 12, 5), (128, 32, 8, 64, 8), (256, 16, 2, 33, 33), (128, 256, 1, 300, 128),
                                           (64, 16, 1, 1, 1)])
def test_accept_moves_rows_as_if_all_were_read_first(d, ps, hkv, Nq, M, fp8):
    """Paths, overlapping places, any order, the same node twice, padding in between."""
    g = gen(5)
    lens = [Nq, Nq + 1, Nq + ps, Nq + 3 * ps + 7]
    B = len(lens)
    per = -(-max(lens) // ps)
    pages = B * per + 2
    cache = api.kv_cache(pages, ps, hkv, d, e4m3=fp8)
    for t in cache:
        if t is not None:
            t.copy_(torch.randint(0, 100, t.shape, generator=g, device=DEV))
    table = torch.randperm(pages, generator=g, device=DEV)[:B * per].view(B, per).to(torch.int32)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    acc = torch.randint(0, Nq, (B, M), generator=g, device=DEV, dtype=torch.int32)
    acc[1] = torch.randperm(Nq, generator=g, device=DEV)[:M].sort().values
    acc[2, M // 2:] = -1
    if M > 2:
        acc[3, 1] = -9
    want = [None if t is None else t.clone() for t in cache]
    for b, n in enumerate(lens):
        slot = lambda i: (int(table[b, (n - Nq + i) // ps]), (n - Nq + i) % ps)
        for j, node in enumerate(acc[b].tolist()):
            if node >= 0:
                (p1, r1), (p0, r0) = slot(j), slot(node)
                for w, t in zip(want, cache):
                    if t is not None:
                        w[p1, :, r1] = t[p0, :, r0]
    api.attn_kv_accept(cache, table, seq, acc, Nq)
    assert api.device_status()[0] == 0
    for w, t in zip(want, cache):
        assert t is None or torch.equal(w.view(torch.uint8), t.view(torch.uint8))


def test_accept_reports_what_it_refuses():
    ps, Nq, M = 16, 6, 4
    for acc, lens, change, site in (
            ([0, 2, 6, 5], 40, None, 0x106), ([0, 2, 3, 5], 5, None, 0x106), ([0, 2, 3, 5], 40, -1, 0x102),
            ([-1, -1, -1, -1], 0, None, None), ([0, 2, 3, 5], 100, None, 0x103)):
        cache = api.kv_cache(6, ps, 2, 64, e4m3=False)
        g = gen(6)
        for t in cache[:2]:
            t.copy_(rand(g, *t.shape))
        table = torch.tensor([[4, 1, 0]], dtype=torch.int32, device=DEV)
        if change is not None:
            table[0, 2] = change                           # tokens 32 to 47: all of the drafts
        before = cache.k.clone()
        api.attn_kv_accept(cache, table, torch.tensor([lens], dtype=torch.int32, device=DEV),
                           torch.tensor([acc], dtype=torch.int32, device=DEV), Nq)
        assert api.device_status() == ((0, 0) if site is None else (-5, site))
        moved = (cache.k != before).any(-1).any(1)         # (page, row)
        at = {(int(p), int(r)) for p, r in moved.nonzero().tolist()}
        if site == 0x106 and lens == 40:
            assert at == {(0, 3), (0, 5)}                  # (nodes 2 and 5 to places 1 and 3)
        elif site == 0x103:                                # cut to 48 tokens: drafts 42 to 47
            assert at == {(0, 11), (0, 12), (0, 13)}
        else:
            assert at == set()


def test_accept_refusals_of_the_binding():
    cache = api.kv_cache(6, 16, 2, 64)
    table, lens = torch.zeros((2, 3), dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    acc = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    for bad in (acc.long(), acc[:1], acc[0], acc.t()):
        with pytest.raises(ValueError, match="accepted"):
            api.attn_kv_accept(cache, table, lens, bad, 8)
    with pytest.raises(api.AttnError, match="accepted of"):
        api.attn_kv_accept(cache, table, lens, acc, 3)
    with pytest.raises(api.AttnError, match="at most"):
        api.attn_kv_accept(cache, table, lens, torch.full((2, 129), -1, dtype=torch.int32, device=DEV), 500)
    api.attn_kv_accept(cache, table[:0], lens[:0], acc[:0], 8)
    api.attn_kv_accept(cache, table, lens, acc[:, :0].contiguous(), 8)
    q = torch.zeros((2, 4, 4, 64), dtype=torch.bfloat16, device=DEV)
    ok = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    for bad in (ok.long(), ok[:1], ok[:, :3], ok.t().contiguous().t(), None):
        with pytest.raises(ValueError, match="parents"):
            api.attn_fwd_paged_tree(q, cache, table, lens, bad)
    with pytest.raises(api.AttnError, match="nodes"):
        api.attn_fwd_paged_tree(torch.zeros((1, 513, 2, 64), dtype=torch.bfloat16, device=DEV), cache, table[:1], lens[:1],
                                torch.full((513,), -1, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_speculative_steps_equal_a_run_without_speculation(fp8, graph):
    """Prompt, then steps of append, tree attention and accept, eager or captured once
    and replayed: the cache then holds bit for bit what appending the accepted
    tokens one after the other gives, and their attention is the causal one's."""
    B, Nq, M, H, hkv, d, ps, steps = 3, 10, 4, 8, 2, 128, 16, 5
    g = gen(50)
    per = 8
    prompt = [5, 30, 17]
    pages = B * per
    order = torch.randperm(pages, generator=g, device=DEV).view(B, per).to(torch.int32)
    cos, sin = ref.tables(256, d, DEV)
    spec, plain = api.kv_cache(pages, ps, hkv, d, e4m3=fp8), api.kv_cache(pages, ps, hkv, d, e4m3=fp8)

    def slots_of(b, at):
        return order[b].long()[at // ps] * ps + at % ps

    for b, n in enumerate(prompt):
        at = torch.arange(n, device=DEV)
        x = rand(g, n, 2 * hkv, d)
        for c in (spec, plain):
            api.attn_kv_append(None, x[:, :hkv], x[:, hkv:], at, slots_of(b, at), c, cos, sin)
    lens = torch.tensor(prompt, device=DEV)
    q, k, v = rand(g, B * Nq, H, d), rand(g, B * Nq, hkv, d), rand(g, B * Nq, hkv, d)
    parents = torch.full((B, Nq), -1, dtype=torch.int32, device=DEV)
    acc = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    pos, slots = torch.zeros(B * Nq, dtype=torch.int64, device=DEV), torch.zeros(B * Nq, dtype=torch.int64, device=DEV)
    seq = torch.zeros(B, dtype=torch.int32, device=DEV)
    turned, out = torch.empty_like(q), torch.empty((B, Nq, H, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((B, H, Nq), device=DEV)
    ws = torch.empty(api.paged_tree_workspace_bytes(B, Nq, H, hkv, d, 0, per, ps), dtype=torch.uint8, device=DEV)

    def step():
        api.attn_kv_append(q, k, v, pos, slots, spec, cos, sin, out_q=turned)
        api.attn_fwd_paged_tree(turned.view(B, Nq, H, d), spec, order, seq, parents, out=out, lse=lse, workspace=ws)
        api.attn_kv_accept(spec, order, seq, acc, Nq)

    captured = None
    for it in range(steps):
        for t in (q, k, v):
            t.copy_(rand(g, *t.shape))
        parents.copy_(random_parents(g, B, Nq, 3))
        paths = [ref.paths(parents[b].tolist()) for b in range(B)]
        depth = torch.tensor([[len(s) - 1 for s in row] for row in paths], device=DEV)
        pos.copy_((lens[:, None] + depth).flatten())
        slots.copy_(torch.stack([slots_of(b, lens[b] + torch.arange(Nq, device=DEV)) for b in range(B)]).flatten())
        seq.copy_(lens + Nq)
        acc.fill_(-1)
        kept = []
        for b in range(B):
            leaf = max(range(Nq), key=lambda i: (len(paths[b][i]) <= M) * len(paths[b][i]))
            kept.append(sorted(paths[b][leaf]))
            acc[b, :len(kept[b])] = torch.tensor(kept[b], dtype=torch.int32, device=DEV)
        if graph and captured is None:
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            saved = [None if t is None else t.clone() for t in spec]
            with torch.cuda.stream(side):
                step()
            torch.cuda.synchronize()
            for t, s in zip(spec, saved):
                if t is not None:
                    t.copy_(s)
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        if captured is not None:
            captured.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert api.device_status()[0] == 0
        for b in range(B):
            at = lens[b] + torch.arange(len(kept[b]), device=DEV)
            rows = b * Nq + torch.tensor(kept[b], device=DEV)
            one = api.attn_kv_append(q[rows], k[rows], v[rows], at, slots_of(b, at), plain, cos, sin)
            n = int(lens[b]) + len(kept[b])
            new = torch.tensor([n], dtype=torch.int32, device=DEV)
            c, cl = api.attn_fwd_paged(one[None], plain, order[b:b + 1], new)
            # (each within its own rounding of the same values; bf16 weights and results)
            o = out[b, torch.tensor(kept[b], device=DEV)]
            assert float((o.float() - c[0].float()).abs().max()) <= 4 * 2.0 ** -8 * float(c.float().abs().max().clamp(min=1))
            assert float((lse[b][:, kept[b]] - cl[0]).abs().max()) <= 1e-4
            x = api.attn_kv_read(spec, order[b:b + 1], new, n)
            y = api.attn_kv_read(plain, order[b:b + 1], new, n)
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        lens = lens + torch.tensor([len(x) for x in kept], device=DEV)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 135])
def test_ranges_of_every_length_in_the_tile_kernel(prefix, d, fp8):
    """A key tile's products leave out its last rows, which hold anything: chains with and
    without the mask, and trees."""
    lens = list(range(40, 57)) + list(range(120, 137)) + [250, 256, 257]
    p = Tree(lens, prefix, 40, 2, 2, d, 64, fp8, seed=24, width=4)
    assert api.paged_plan(len(lens), 40, 2, 2, d, prefix, p.table.shape[1], 64).own_kernel == "tile"
    got = []
    for stale in (0x7f, 0x7e):                          # NaN, and large values
        for b, n in enumerate(lens):                    # the rest of a sequence's last page
            page, row = int(p.table[b, (n - 1) // 64]), (n - 1) % 64 + 1
            for x in (p.cache.k, p.cache.v):
                x[page, :, row:] = stale if fp8 else (NAN if stale == 0x7f else 1e38)
            if fp8:
                for x in (p.cache.k_scale, p.cache.v_scale):
                    x[page, :, row:] = NAN if stale == 0x7f else 1e30
        now = []
        for causal in (True, False):
            o, lse = Problem.run(p, causal=causal)
            Problem.check(p, o, lse, causal=causal)
            now += [o, lse]
        o, lse = p.run()
        p.check(o, lse)
        got.append(now + [o, lse])
    assert all(torch.equal(a, b) for a, b in zip(*got))
