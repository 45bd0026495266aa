"""The paged cache's entries without a GPU: argument checks (before any launch),
workspace sizes and the Python binding's refusals."""
import ctypes

import pytest
import torch

from exact_attention_71_gb300 import api, build

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: the checks fail first
ODD = ctypes.c_void_p((1 << 20) + 4)
BF16, E4M3 = api.CACHE_BF16, api.CACHE_E4M3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.library()


def write(lib, k=FAKE, v=FAKE, ks=1024, vs=1024, slots=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, T=4, hkv=8, d=128,
          pages=10, ps=16, dtype=E4M3):
    return lib.attn_kv_write(k, v, ks, vs, slots, kc, vc, ksc, vsc, T, hkv, d, pages, ps, dtype, None)


def read(lib, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, table=FAKE, stride=4, max_pages=4, lens=FAKE, k=FAKE, v=FAKE, B=2,
         N=50, hkv=8, d=128, pages=10, ps=16, dtype=E4M3):
    return lib.attn_kv_read(kc, vc, ksc, vsc, table, stride, max_pages, lens, k, v, B, N, hkv, d, pages, ps, dtype, None)


def attend(lib, q=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, pre=FAKE, prefix=100, table=FAKE, stride=4, max_pages=4,
           lens=FAKE, o=FAKE, lse=FAKE, B=2, Nq=1, H=16, hkv=8, d=128, pages=10, ps=16, dtype=E4M3, causal=1, scale=0.0,
           ws=FAKE, wsb=1 << 30):
    return lib.attn_fwd_paged(q, kc, vc, ksc, vsc, pre, prefix, table, stride, max_pages, lens, o, lse, B, Nq, H, hkv, d,
                              pages, ps, dtype, causal, scale, ws, wsb, None)


def test_cache_arguments_are_checked_by_every_entry(lib):
    for f in (write, read, attend):
        for d in (32, 96, 192, 512):
            assert f(lib, d=d) == -2
        assert b"head_dim" in lib.attn_last_error_string()
        for ps in (0, 8, 48, 512, -16):
            assert f(lib, ps=ps) == -2
        assert b"page_size" in lib.attn_last_error_string()
        assert f(lib, dtype=2) == -1 and b"cache_dtype" in lib.attn_last_error_string()
        assert f(lib, hkv=0) == -1
        assert f(lib, pages=-1) == -1
        assert f(lib, kc=None) == -1 and f(lib, vc=None) == -1
        assert f(lib, ksc=None) == -1 and b"scale" in lib.attn_last_error_string()
        assert f(lib, kc=ODD) == -1 and b"aligned" in lib.attn_last_error_string()


def test_write_arguments(lib):
    assert write(lib, T=-1) == -1
    assert write(lib, T=0) == 0
    assert write(lib, k=None) == -1 and write(lib, slots=None) == -1
    assert write(lib, v=ODD) == -1
    assert write(lib, slots=ODD) == -1 and b"slots" in lib.attn_last_error_string()
    assert write(lib, ks=1020) == -1 and b"multiples of 8" in lib.attn_last_error_string()
    assert write(lib, T=1 << 28, hkv=8) == -1 and b"too large" in lib.attn_last_error_string()


def test_read_arguments(lib):
    assert read(lib, B=0) == 0 and read(lib, N=0) == 0
    assert read(lib, B=-1) == -1 and read(lib, max_pages=-1) == -1
    assert read(lib, stride=3) == -1 and b"table_stride" in lib.attn_last_error_string()
    assert read(lib, table=None) == -1 and read(lib, lens=None) == -1 and read(lib, k=None) == -1
    assert read(lib, max_pages=1 << 27, stride=1 << 27) == -1 and b"2^30" in lib.attn_last_error_string()
    assert read(lib, B=70000) == -1


def test_attention_arguments(lib):
    assert attend(lib, B=0) == 0 and attend(lib, Nq=0) == 0 and attend(lib, H=0) == 0
    assert attend(lib, H=12) == -1 and b"divide" in lib.attn_last_error_string()
    assert attend(lib, B=-1) == -1 and attend(lib, prefix=-1) == -1
    assert attend(lib, prefix=(1 << 30) + 1) == -1 and b"2^30" in lib.attn_last_error_string()
    assert attend(lib, pre=None) == -1
    assert attend(lib, q=None) == -1 and attend(lib, o=None) == -1 and attend(lib, lse=None) == -1
    assert attend(lib, q=ctypes.c_void_p((1 << 20) + 8)) == -1
    assert attend(lib, ws=None) == -1
    assert attend(lib, ws=ctypes.c_void_p((1 << 20) + 16)) == -1 and b"256-byte" in lib.attn_last_error_string()
    need = lib.attn_fwd_paged_workspace_size(2, 1, 16, 8, 128, 100, 4, 16)
    assert need > 0
    assert attend(lib, wsb=need - 1) == -1 and b"smaller" in lib.attn_last_error_string()


def test_workspace_sizes(lib):
    size = lib.attn_fwd_paged_workspace_size
    # invalid and empty problems need nothing
    assert size(-1, 1, 16, 8, 128, 0, 4, 16) == 0
    assert size(2, 1, 12, 8, 128, 0, 4, 16) == 0
    assert size(2, 1, 16, 8, 96, 0, 4, 16) == 0
    assert size(0, 1, 16, 8, 128, 100, 4, 16) == 0
    # one part: the kernel writes the result itself
    assert size(600, 1, 16, 8, 128, 0, 4, 16) == 0
    assert size(2, 1, 16, 8, 128, 0, 0, 16) == 0
    # parts x rows of (d + 1) floats, the two arrays 256-byte aligned; at least one
    # part of the prefix and one of the own tokens
    up = lambda x: (x + 255) // 256 * 256
    rows, d = 2 * 1 * 16, 128
    need = size(2, 1, 16, 8, d, 100, 4, 16)
    parts = [n for n in range(2, 513) if up(n * rows * d * 4) + up(n * rows * 4) == need]
    assert len(parts) == 1
    # it does not depend on anything but its arguments, and is bounded: at most 256
    # ranges of either segment
    for args in ((1, 1, 1, 1, 64, 1 << 20, 1 << 12, 256), (128, 5, 32, 8, 128, 16384, 64, 16), (3, 512, 16, 2, 256, 999, 9, 64)):
        rows = args[0] * args[1] * args[2]
        assert size(*args) == size(*args) <= up(512 * rows * args[4] * 4) + up(512 * rows * 4)


def test_binding_refuses_tensors_that_are_not_what_it_says():
    """On CPU tensors every call stops in the binding (the cache has to be on a
    GPU); nothing reaches the library."""
    cache = api.KVCache(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_kv_write(x, x, torch.zeros(1, dtype=torch.int64), cache)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_kv_read(cache, table, lens, 4)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_fwd_paged(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), cache, table, lens)
