"""attn_rope, attn_kv_append, attn_fwd_paged_tree and attn_kv_accept without a GPU:
argument checks (before any launch), workspace sizes, the binding's refusals, and the
tests' own plain forms."""
import ctypes

import pytest
import torch

from exact_attention_71_gb300 import api, build
from tests import rope_ref

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: the checks fail first
FAR = ctypes.c_void_p(1 << 40)
ODD = ctypes.c_void_p((1 << 20) + 4)
BF16, E4M3 = api.CACHE_BF16, api.CACHE_E4M3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.library()


def rope(lib, q=FAKE, qs=1024, qo=FAR, qos=1024, k=None, ks=0, ko=None, kos=0, pos=FAKE, stride=4, axes=1, pair=None, cos=FAKE,
         sin=FAKE, rows=100, rot=128, T=4, period=0, H=8, hkv=0, d=128):
    return lib.attn_rope(q, qs, qo, qos, k, ks, ko, kos, pos, stride, axes, pair, cos, sin, rows, rot, 0, 0, T, period, H, hkv,
                         d, None)


def append(lib, q=FAKE, qs=1024, qo=FAR, qos=1024, k=FAKE, v=FAKE, ks=1024, vs=1024, pos=FAKE, stride=4, axes=1, pair=None,
           cos=FAKE, sin=FAKE, rows=100, rot=128, slots=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, T=4, H=8, hkv=8, d=128,
           pages=10, ps=16, dtype=E4M3):
    return lib.attn_kv_append(q, qs, qo, qos, k, v, ks, vs, pos, stride, axes, pair, cos, sin, rows, rot, 0, slots, kc, vc, ksc,
                              vsc, T, H, hkv, d, pages, ps, dtype, None)


def tree(lib, q=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, pre=FAKE, prefix=100, table=FAKE, stride=4, max_pages=4, lens=FAKE,
         parents=FAKE, pstride=8, o=FAKE, lse=FAKE, B=2, Nq=8, H=16, hkv=8, d=128, pages=10, ps=16, dtype=E4M3, ws=FAKE,
         wsb=1 << 30):
    return lib.attn_fwd_paged_tree(q, kc, vc, ksc, vsc, pre, prefix, table, stride, max_pages, lens, parents, pstride, o, lse,
                                   B, Nq, H, hkv, d, pages, ps, dtype, 0.0, ws, wsb, None)


def accept(lib, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, table=FAKE, stride=4, max_pages=4, lens=FAKE, acc=FAKE, B=2, Nq=8, M=4,
           hkv=8, d=128, pages=10, ps=16, dtype=E4M3):
    return lib.attn_kv_accept(kc, vc, ksc, vsc, table, stride, max_pages, lens, acc, B, Nq, M, hkv, d, pages, ps, dtype, None)


def error(lib):
    return lib.attn_last_error_string()


def test_cache_arguments_are_checked_by_every_entry(lib):
    for f in (append, tree, accept):
        for d in (32, 96, 192, 512):
            assert f(lib, d=d) == -2
        assert b"head_dim" in error(lib)
        for ps in (0, 8, 48, 512, -16):
            assert f(lib, ps=ps) == -2
        assert f(lib, dtype=2) == -1 and f(lib, hkv=0) == -1 and f(lib, pages=-1) == -1
        assert f(lib, kc=None) == -1 and f(lib, vc=None) == -1
        assert f(lib, ksc=None) == -1 and b"scale" in error(lib)
        assert f(lib, kc=ODD) == -1 and b"aligned" in error(lib)


def test_rotation_arguments(lib):
    for f in (rope, append):
        for rot in (0, 8, 24, 144, -16):
            assert f(lib, rot=rot) == -2
        assert b"rotary" in error(lib)
        assert f(lib, axes=0) == -2 and f(lib, axes=5) == -2 and b"axes" in error(lib)
        assert f(lib, axes=2) == -1 and b"pair_axis" in error(lib)
        assert f(lib, axes=2, pair=bytes([0, 1] * 31 + [0, 2])) == -1 and b"pair 63" in error(lib)
        assert f(lib, axes=1, pair=bytes([0] * 63 + [1])) == -1
        assert f(lib, cos=None) == -1 and f(lib, sin=None) == -1 and b"table" in error(lib)
        assert f(lib, cos=ODD) == -1 and b"aligned" in error(lib)
        assert f(lib, rows=-1) == -1 and f(lib, pos=ODD) == -1 and b"positions" in error(lib)
        assert f(lib, T=-1) == -1 and f(lib, H=-1) == -1
        assert f(lib, T=0) == 0
        assert f(lib, T=1 << 28) == -1 and b"too large" in error(lib)
        assert f(lib, q=None) == -1 and f(lib, qo=None) == -1 and f(lib, qo=ODD) == -1
        assert f(lib, qs=1020) == -1 and b"multiples of 8" in error(lib)
        assert f(lib, qs=-1024) == -1 and b"negative" in error(lib)
        assert f(lib, qos=1016) == -1 and b"overlap" in error(lib)
        # output rows that meet the input's and are not the same rows
        assert f(lib, qo=FAKE, qos=2048) == -1 and b"overlaps" in error(lib)
        assert f(lib, qo=ctypes.c_void_p((1 << 20) + 2048)) == -1 and b"overlaps" in error(lib)
        assert f(lib, qs=2048, qos=2048, qo=ctypes.c_void_p((1 << 20) + 2032)) == -1
    assert rope(lib, d=96) == -2
    assert rope(lib, pos=None, rows=3) == -1 and b"shorter" in error(lib)
    assert rope(lib, pos=None, axes=2, pair=bytes([0, 1] * 32)) == -1 and b"positions" in error(lib)
    assert rope(lib, period=-1) == -1
    assert rope(lib, H=0) == 0
    assert rope(lib, k=FAKE, ks=1024, ko=FAR, kos=1024, hkv=8) == -1 and b"written" in error(lib)
    assert append(lib, pos=None) == -1 and append(lib, k=None) == -1 and append(lib, v=ODD) == -1
    assert append(lib, slots=None) == -1 and append(lib, slots=ODD) == -1 and b"slots" in error(lib)
    assert append(lib, ks=1020) == -1 and append(lib, vs=-1024) == -1
    assert append(lib, k=FAR) == -1 and b"new keys" in error(lib)


def test_tree_arguments(lib):
    assert tree(lib, B=0) == 0 and tree(lib, Nq=0) == 0 and tree(lib, H=0) == 0
    assert tree(lib, H=12) == -1 and b"divide" in error(lib)
    assert tree(lib, Nq=513, pstride=513) == -2 and b"nodes" in error(lib)
    assert tree(lib, parents=None) == -1 and tree(lib, parents=ctypes.c_void_p((1 << 20) + 2)) == -1
    assert tree(lib, pstride=7) == -1 and b"parents_stride" in error(lib)
    assert tree(lib, pre=None) == -1 and tree(lib, lens=None) == -1 and tree(lib, table=None) == -1
    assert tree(lib, q=None) == -1 and tree(lib, o=None) == -1 and tree(lib, lse=None) == -1
    assert tree(lib, stride=3) == -1 and tree(lib, prefix=-1) == -1
    need = lib.attn_fwd_paged_tree_workspace_size(2, 8, 16, 8, 128, 100, 4, 16)
    assert tree(lib, ws=None) == -1 and tree(lib, wsb=need - 1) == -1 and b"smaller" in error(lib)
    assert tree(lib, ws=ctypes.c_void_p((1 << 20) + 16)) == -1


def test_tree_workspace_is_the_attentions(lib):
    size, plain = lib.attn_fwd_paged_tree_workspace_size, lib.attn_fwd_paged_workspace_size
    for args in ((2, 8, 16, 8, 128, 100, 4, 16), (3, 512, 16, 2, 256, 999, 9, 64), (1, 5, 4, 4, 64, 0, 4096, 16)):
        assert size(*args) == plain(*args) > 0
    assert size(600, 1, 16, 8, 128, 0, 4, 16) == 0         # one part: written without a join
    assert size(2, 513, 16, 8, 128, 0, 4, 16) == 0 and size(0, 8, 16, 8, 128, 0, 4, 16) == 0
    assert size(2, 8, 12, 8, 128, 0, 4, 16) == 0


def test_accept_arguments(lib):
    assert accept(lib, B=0) == 0 and accept(lib, M=0) == 0
    assert accept(lib, B=-1) == -1 and accept(lib, Nq=-1) == -1 and accept(lib, M=-1) == -1
    assert accept(lib, M=9) == -1 and b"accepted of" in error(lib)
    assert accept(lib, Nq=200, M=129) == -2 and b"at most" in error(lib)
    assert accept(lib, acc=None) == -1 and accept(lib, acc=ctypes.c_void_p((1 << 20) + 2)) == -1
    assert accept(lib, lens=None) == -1 and accept(lib, table=None) == -1 and accept(lib, stride=3) == -1
    assert accept(lib, B=1 << 28) == -1 and b"too large" in error(lib)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    cos = torch.ones(4, 32)
    n, one = torch.zeros(1, dtype=torch.int64), torch.ones(1, dtype=torch.int32)
    cache = api.KVCache(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_rope(x, x, cos, cos)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_kv_append(x, x, x, n, n, cache, cos, cos)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_fwd_paged_tree(x[None], cache, table, one, table[:, :1])
    with pytest.raises(ValueError, match="parents"):
        api.attn_fwd_paged_tree(x[None], cache, table, one, None)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_kv_accept(cache, table, one, table[:, :1], 1)


def test_plain_paths():
    assert rope_ref.paths([-1, 0, 0, 2]) == [{0}, {0, 1}, {0, 2}, {0, 2, 3}]
    assert rope_ref.paths([1, -1, -2, 2, 4, 9, 7, 6]) == [{0, 1}, {1}, None, None, None, None, None, None]


def test_plain_rotation_keeps_lengths_and_its_transpose_undoes_it():
    g = torch.Generator().manual_seed(0)
    cos, sin = rope_ref.tables(50, 48, "cpu")
    pos = torch.randint(0, 50, (2, 7), generator=g)
    axis = tuple(i % 2 for i in range(24))
    x = torch.randn(7, 3, 64, generator=g, dtype=torch.float64)
    for il in (False, True):
        c, s = rope_ref.gather(cos, sin, pos, axis)
        y, _ = rope_ref.turn(x, c, s, 48, il)
        back, _ = rope_ref.turn(y, *rope_ref.gather(cos, sin, pos, axis, True), 48, il)
        # (float32 tables: cos^2 + sin^2 is 1 within 2^-22)
        assert float((back - x).abs().max()) <= 2.0 ** -20 and torch.equal(y[..., 48:], x[..., 48:])
