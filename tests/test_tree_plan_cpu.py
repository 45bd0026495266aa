"""How calls of attn_fwd_paged_tree are cut up (host arithmetic), and that the GPU tests'
shapes between them reach every kernel in every mode."""
import ctypes

import pytest

from exact_attention_71_gb300 import api, build
from tests import test_gpu_tree as tree
from tests import test_gpu_tree_modes as modes


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return api.library()


SHAPES = [s[:-1] for s in tree.SHAPES + tree.EMPTIES] + modes.MODES


def chain_rows(d):
    """Rows of a key/value head that a chain's streaming kernel takes at most."""
    return 16 if d == 256 else 32


def modes_of(shape):
    """(head dim, kernel, rows of a streaming CTA or one / several row tiles, segment,
    written without a join, more rows than a chain's) of a call."""
    p, out = modes.plan(shape), set()
    lens, _, Nq, H, hkv, d, _ = shape
    rows = Nq * (H // hkv)
    for segment, kernel, tiles, n in (("prefix", p.prefix_kernel, p.prefix_row_tiles, rows * len(lens)),
                                      ("own", p.own_kernel, p.own_row_tiles, rows)):
        if kernel == "stream":
            out.add((d, kernel, p.stream_rows, segment, p.direct, n > chain_rows(d)))
        elif kernel == "tile":
            out.add((d, kernel, "one" if tiles == 1 else "several", segment, p.direct, None))
    return out


def test_the_gpu_tests_reach_every_kernel_in_every_mode():
    want = {(d, kernel, rows, segment, direct, more)
            for d in (64, 128, 256)
            for kernel, all_rows in (("stream", ((8, False), (16, False), (16, True))), ("tile", (("one", None), ("several", None))))
            for rows, more in all_rows
            for segment, direct in (("prefix", False), ("own", False), ("own", True))}
    have = set().union(*map(modes_of, SHAPES))
    assert want <= have, sorted(map(str, want - have))


def test_the_gpu_tests_reach_the_last_bit_of_a_path_and_every_join():
    """32 nodes in the streaming kernel at each head dim; prefix and own tokens in
    either kernel beside one another."""
    full = {s[5] for s in modes.MODES if s[2] == 32 and modes.plan(s).own_kernel == "stream"}
    assert full == {64, 128, 256}
    pairs = {(p.prefix_kernel, p.own_kernel) for p in map(modes.plan, SHAPES)}
    assert pairs == {(None, "stream"), (None, "tile"), ("stream", "stream"), ("tile", "stream"), ("tile", "tile")}


def test_trees_stream_where_chains_do_not():
    args = (4, 8, 32, 8, 128, 512, 7, 16)
    chain, trees = api.paged_plan(*args), api.paged_tree_plan(*args)
    assert (chain.prefix_kernel, chain.own_kernel) == ("tile", "stream")
    assert (trees.prefix_kernel, trees.own_kernel) == ("stream", "stream")
    assert api.paged_workspace_bytes(*args) != api.paged_tree_workspace_bytes(*args)
    # as chains: 33 nodes, many rows, long own tokens
    for args in ((2, 33, 4, 4, 64, 0, 8, 16), (64, 16, 32, 8, 128, 8192, 16, 64), (1, 16, 32, 8, 128, 0, 100, 64)):
        assert api.paged_plan(*args)[:2] == api.paged_tree_plan(*args)[:2]


def test_plan_and_workspace_agree():
    up = lambda x: (x + 255) // 256 * 256
    for shape in SHAPES:
        lens, prefix, Nq, H, hkv, d, ps = shape
        p = modes.plan(shape)
        n = (p.prefix_parts + p.own_parts) * len(lens) * Nq * H
        assert p.direct == (p.prefix_parts + p.own_parts == 1)
        per = max(1, -(-max(lens + [1]) // ps)) + 1
        want = 0 if p.direct else up(n * d * 4) + up(n * 4)
        assert api.paged_tree_workspace_bytes(len(lens), Nq, H, hkv, d, prefix, per, ps) == want


def test_refused_sizes_have_no_plan(lib):
    assert api.paged_tree_plan(0, 1, 4, 2, 64, 0, 1, 16) is None
    assert api.paged_tree_plan(1, 1, 3, 2, 64, 0, 1, 16) is None
    assert api.paged_tree_plan(1, 513, 4, 2, 64, 0, 1, 16) is None and api.paged_plan(1, 513, 4, 2, 64, 0, 1, 16) is not None
    assert api.paged_tree_plan(1, 512, 4, 2, 64, 0, 1, 16) is not None
    buf = (ctypes.c_int * 8)()
    assert lib.attn_fwd_paged_tree_plan(1, 1, 4, 2, 64, 0, 1, 16, ctypes.cast(buf, ctypes.c_void_p), 7) == 0
    assert lib.attn_fwd_paged_tree_plan(1, 1, 4, 2, 64, 0, 1, 16, None, 8) == 0
