"""attn_kv_accept where a sequence is longer than its table: nothing of it is moved."""
import pytest
import torch

from exact_attention_71_gb300 import api
from tests.test_gpu_paged import gen, rand

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M", [4, 12, 30])               # rows in registers (8, 16), in shared memory
@pytest.mark.parametrize("over", [1, 52, (1 << 31) - 49])
def test_no_row_of_a_sequence_beyond_its_table_is_moved(over, M, fp8):
    """The drafts of a sequence of n tokens are n - Nq to n - 1, whatever its table holds:
    tokens before them are context and keep every byte.  Sequences that fit, also those
    that fill their table, move as always."""
    ps, per, Nq, hkv, d = 16, 3, 32, 2, 64
    room = per * ps
    lens = [room, room + over, 40]
    g = gen(6)
    cache = api.kv_cache(3 * per, ps, hkv, d, e4m3=fp8)
    for t in cache:
        if t is not None:
            t.copy_(rand(g, *t.shape) if t.dtype == torch.bfloat16 else torch.randint(1, 100, t.shape, generator=g, device=DEV))
    table = torch.randperm(3 * per, generator=g, device=DEV).to(torch.int32).view(3, per)
    acc = torch.arange(M, dtype=torch.int32, device=DEV) + 2
    acc[0] = 0
    acc = acc.repeat(3, 1)
    want = [None if t is None else t.clone() for t in cache]
    for b in (0, 2):
        at = lambda node: lens[b] - Nq + node
        slot = lambda i: (int(table[b, i // ps]), i % ps)
        for j in range(M):
            (p1, r1), (p0, r0) = slot(at(j)), slot(at(int(acc[b, j])))
            for w, t in zip(want, cache):
                if w is not None:
                    w[p1, :, r1] = t[p0, :, r0]
    api.attn_kv_accept(cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), acc, Nq)
    assert api.device_status() == (-5, 0x103)
    for w, t in zip(want, cache):
        assert w is None or torch.equal(w.view(torch.uint8), t.view(torch.uint8))


def test_a_table_of_no_columns_moves_nothing():
    cache = api.kv_cache(2, 16, 1, 64, e4m3=False)
    cache.k.copy_(rand(gen(7), *cache.k.shape))
    before = cache.k.clone()
    acc = torch.tensor([[2, 3]], dtype=torch.int32, device=DEV)
    api.attn_kv_accept(cache, torch.zeros((1, 0), dtype=torch.int32, device=DEV), torch.tensor([9], dtype=torch.int32, device=DEV),
                       acc, 4)
    assert api.device_status() == (-5, 0x103)
    assert torch.equal(cache.k, before)
