"""How paged attention calls are cut up (host arithmetic), and that the GPU tests'
shapes between them reach every kernel in every mode."""
import ctypes

import pytest

from exact_attention_71_gb300 import api, build
from tests import test_gpu_paged as paged
from tests import test_gpu_paged_modes as modes


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return api.library()


def modes_of(shape):
    """(head dim, kernel, rows of a streaming CTA or one / several row tiles, segment,
    written without a join) of a call."""
    p, d, out = modes.plan(shape), shape[5], set()
    for segment, kernel, tiles in (("prefix", p.prefix_kernel, p.prefix_row_tiles), ("own", p.own_kernel, p.own_row_tiles)):
        if kernel == "stream":
            out.add((d, kernel, p.stream_rows, segment, p.direct))
        elif kernel == "tile":
            out.add((d, kernel, "one" if tiles == 1 else "several", segment, p.direct))
    return out


def test_the_gpu_tests_reach_every_kernel_in_every_mode():
    want = {(d, kernel, rows, segment, direct)
            for d in (64, 128, 256)
            for kernel, all_rows in (("stream", (8, 16)), ("tile", ("one", "several")))
            for rows in all_rows
            for segment, direct in (("prefix", False), ("own", False), ("own", True))}
    have = set().union(*map(modes_of, paged.SHAPES + modes.MODES))
    assert want <= have, sorted(map(str, want - have))


def test_many_ranges_are_joined():
    parts = {p.prefix_parts + p.own_parts for p in map(modes.plan, paged.SHAPES + modes.MODES)}
    assert any(n > 128 for n in parts) and any(32 < n <= 128 for n in parts) and 2 in parts


def test_plan_and_workspace_agree():
    up = lambda x: (x + 255) // 256 * 256
    for shape in paged.SHAPES + modes.MODES:
        lens, prefix, Nq, H, hkv, d, ps = shape
        args = (len(lens), Nq, H, hkv, d, prefix, max(1, -(-max(lens + [1]) // ps)) + 1, ps)
        p = api.paged_plan(*args)
        n = (p.prefix_parts + p.own_parts) * len(lens) * Nq * H
        assert p.direct == (p.prefix_parts + p.own_parts == 1)
        assert api.paged_workspace_bytes(*args) == (0 if p.direct else up(n * d * 4) + up(n * 4))


def test_refused_sizes_have_no_plan(lib):
    assert api.paged_plan(0, 1, 4, 2, 64, 0, 1, 16) is None
    assert api.paged_plan(1, 1, 3, 2, 64, 0, 1, 16) is None
    assert api.paged_plan(1, 1, 4, 2, 96, 0, 1, 16) is None
    assert api.paged_plan(1, 1, 4, 2, 64, -1, 1, 16) is None
    buf = (ctypes.c_int * 8)()
    assert lib.attn_fwd_paged_plan(1, 1, 4, 2, 64, 0, 1, 16, ctypes.cast(buf, ctypes.c_void_p), 7) == 0
    assert lib.attn_fwd_paged_plan(1, 1, 4, 2, 64, 0, 1, 16, None, 8) == 0


def ctas(args):
    """CTAs of a call's two launches, from its plan."""
    B, Nq, H, hkv, d, prefix, pages, ps = args
    p = api.paged_plan(*args)
    if p is None:
        return None
    up = lambda a, b: -(-a // b)
    groups = lambda tiles: tiles if d == 256 else up(tiles, 2)
    rows = Nq * (H // hkv)
    tile = stream = 0
    if p.prefix_kernel == "tile":
        tile += hkv * groups(p.prefix_row_tiles) * p.prefix_parts
    elif p.prefix_kernel == "stream":
        stream += hkv * up(B * rows, p.stream_rows) * p.prefix_parts
    if p.own_kernel == "tile":
        tile += B * hkv * groups(p.own_row_tiles) * p.own_parts
    else:
        stream += B * hkv * up(rows, p.stream_rows) * p.own_parts
    return max(tile, stream)


def test_large_problems_have_fewer_than_2_to_the_31_ctas():
    """Block indices are ints: the sizes that are accepted stay below, with many
    ranges and many sequences together."""
    most = 0
    for d in (64, 128, 256):
        for log_b in range(0, 31, 2):
            for hkv in (1, 8, 1 << 10):
                for Nq, group in ((1, 1), (1, 8), (5, 4), (64, 4), (512, 1)):
                    for prefix, pages in ((0, 1), (0, 1 << 22), (1 << 30, 1 << 22), (1 << 20, 1 << 10)):
                        n = ctas((1 << log_b, Nq, hkv * group, hkv, d, prefix, pages, 256))
                        if n is not None:
                            most = max(most, n)
                            assert n < 1 << 31
    assert most > 1 << 28                              # (the largest accepted ones are among these)


def test_more_sequences_than_a_grid_dimension_has(lib):
    """The attention's grids have one dimension; reading back is a grid row a
    sequence, and says so."""
    assert api.paged_plan(70000, 1, 1, 1, 64, 0, 1, 16) is not None
    fake = ctypes.c_void_p(1 << 20)
    assert lib.attn_kv_read(fake, fake, fake, fake, fake, 4, 4, fake, fake, fake, 70000, 5, 1, 64, 10, 16, 1, None) == -1
    assert b"too large" in lib.attn_last_error_string()
    assert api.paged_plan(1 << 30, 2, 1, 1, 64, 0, 1, 16) is None


def test_the_scales_of_a_bf16_cache_are_ignored(lib):
    """Whatever their pointers are; those of an e4m3 cache have to be aligned."""
    fake, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
    write = lambda dtype: lib.attn_kv_write(fake, fake, 64, 64, fake, fake, fake, odd, odd, 0, 1, 64, 4, 16, dtype, None)
    assert write(api.CACHE_BF16) == 0
    assert write(api.CACHE_E4M3) == -1 and b"aligned" in lib.attn_last_error_string()
