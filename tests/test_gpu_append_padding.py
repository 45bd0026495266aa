"""attn_kv_append through the C entry with padding behind the last token, which needs no
positions: the array ends where the tokens do."""
import ctypes

import pytest
import torch

from exact_attention_71_gb300 import api
from tests import rope_ref as ref
from tests.test_gpu_paged import filled_cache, gen, rand
from tests.test_gpu_rope_rows import sections

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("T, tokens", [(1, 0), (40, 33), (5000, 4097)])
def test_padding_behind_the_last_token_needs_no_positions(T, tokens, axes, fp8):
    """The last axis's array is as long as the tokens; what stands behind it (in the same
    allocation) would be reported if it were taken for a position."""
    H, hkv, d, ps = 4, 2, 128, 16
    g = gen(9)
    x = rand(g, T, H + 2 * hkv, d)
    cos, sin = ref.tables(700, d, DEV)
    slots = torch.randperm((T // ps + 2) * ps, generator=g, device=DEV)[:T]
    slots[tokens:] = -1
    given = torch.full((axes * T,), 1 << 40, dtype=torch.int64, device=DEV)
    pos = torch.zeros((axes, T), dtype=torch.int64, device=DEV)
    pos[:, :tokens] = torch.randint(0, 700, (axes, tokens), generator=g, device=DEV)
    given[:(axes - 1) * T] = pos[:-1].flatten()
    given[(axes - 1) * T:(axes - 1) * T + tokens] = pos[-1, :tokens]
    pair = sections(d // 2, axes, True)
    caches = [filled_cache(T // ps + 2, ps, hkv, d, fp8) for _ in range(2)]
    want = api.attn_kv_append(x[:, :H], x[:, H:H + hkv], x[:, H + hkv:], pos if axes > 1 else pos[0], slots, caches[0], cos, sin,
                              pair if axes > 1 else None)
    assert api.device_status()[0] == 0
    got = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    q, k, v = x[:, :H], x[:, H:H + hkv], x[:, H + hkv:]
    c = caches[1]
    scales = [None if t is None else t.data_ptr() for t in (c.k_scale, c.v_scale)]
    stride = x.stride(0)
    rc = api.library().attn_kv_append(
        q.data_ptr(), stride, got.data_ptr(), H * d, k.data_ptr(), v.data_ptr(), stride, stride, given.data_ptr(), T, axes,
        bytes(pair) if axes > 1 else None, cos.data_ptr(), sin.data_ptr(), 700, d, 0, slots.data_ptr(), c.k.data_ptr(), c.v.data_ptr(),
        *scales, T, H, hkv, d, c.k.shape[0], ps, api.CACHE_E4M3 if fp8 else api.CACHE_BF16,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0 and api.device_status() == (0, 0)
    assert torch.equal(got, want) and bool((got[tokens:] == 0).all())
    for a, b in zip(*caches):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
