"""The paged key/value cache on the GPU: writing, reading back and the attention
behind a shared prefix, against plain forms in 64 bits."""
import math

import pytest
import torch

from exact_attention_71_gb300 import api
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def filled_cache(pages, ps, hkv, d, fp8, value=None):
    """A cache whose every row holds `value` (NaN rows unless said otherwise):
    what is not written must not be seen."""
    c = api.kv_cache(pages, ps, hkv, d, e4m3=fp8)
    if fp8:
        c.k.fill_(0x7f)
        c.v.fill_(0x7f)
        c.k_scale.fill_(NAN)
        c.v_scale.fill_(NAN)
    else:
        c.k.fill_(NAN if value is None else value)
        c.v.fill_(NAN if value is None else value)
    return c


def code_values(c):
    return c.view(torch.float8_e4m3fn).double()


def cache_rows(cache, n):
    """(pages, H_kv, ps, d) values of k or v as float64."""
    x = getattr(cache, n)
    if x.dtype == torch.bfloat16:
        return x.double()
    return code_values(x) * getattr(cache, n + "_scale").double()[..., None]


class Problem:
    """Random sequences written to a cache through attn_kv_write."""

    def __init__(self, lens, prefix, Nq, H, hkv, d, ps, fp8, seed=0, kscale=1.0, extra_pages=2, spread=None):
        g = gen(seed)
        self.lens, self.prefix, self.Nq = lens, prefix, Nq
        B = len(lens)
        per = max(1, -(-max(lens + [1]) // ps)) + 1
        shared = -(-prefix // ps)
        pages = shared + B * per + extra_pages
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        self.prefix_table = order[:shared].contiguous()
        self.table = order[shared:shared + B * per].view(B, per).contiguous()
        self.cache = filled_cache(pages, ps, hkv, d, fp8)
        self.k = [rand(g, n, hkv, d, scale=kscale) for n in [prefix] + lens]
        self.v = [rand(g, n, hkv, d) for n in [prefix] + lens]
        for b, (k, v) in enumerate(zip(self.k, self.v)):
            t = self.prefix_table if b == 0 else self.table[b - 1]
            n = torch.arange(len(k), device=DEV)
            slots = t.long()[n // ps] * ps + n % ps if len(k) else n
            api.attn_kv_write(k, v, slots, self.cache)
        # Entries past a sequence's last token are never read.
        for b, n in enumerate(lens):
            self.table[b, -(-n // ps):] = -(1 << 30)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.q = rand(g, B, Nq, H, d)
        self.fp8, self.d, self.hkv, self.ps = fp8, d, hkv, ps

    def values(self, n, b):
        """float64 keys or values of sequence b (-1: the prefix) as the cache holds them."""
        x = getattr(self, n)[b + 1]
        if not self.fp8:
            return x.double()
        c, s = ref.quantise(x)
        return c * s.double()[..., None]

    def run(self, causal=True, **kw):
        return api.attn_fwd_paged(self.q, self.cache, self.table, self.seq_lens, self.prefix_table, self.prefix,
                                  causal=causal, **kw)

    def check(self, o, lse, causal=True, scale=None):
        assert api.device_status()[0] == 0
        for b, n in enumerate(self.lens):
            k = torch.cat([self.values("k", -1), self.values("k", b)])
            v = torch.cat([self.values("v", -1), self.values("v", b)])
            sees = [self.prefix + (max(0, n - self.Nq + 1 + i) if causal else n) for i in range(self.Nq)]
            want, wl, spread, size = ref.attend(self.q[b].double(), k, v, sees, scale)
            to, tl = ref.tolerances(want, wl, spread, size, self.d)
            err = (o[b].double() - want).abs()
            within = bool((err <= to).all())
            assert within, (b, float((err - to).max()), float(err.max()))
            empty = torch.isinf(wl)
            assert torch.equal(torch.isinf(lse[b]) & (lse[b] < 0), empty)
            dl = (lse[b].double() - wl).abs()[~empty]
            within = bool((dl <= tl[~empty]).all())
            assert within, (b, float(dl.max()))


# Every kernel and mode: few rows (streaming kernel) and many (tile kernel: one row
# tile or pairs of them, an odd number of tiles), both over the prefix and over own
# tokens; ranges that end inside a page, a key tile, a step; one part and many.
SHAPES = [
    # lens, prefix, Nq, H, H_kv, d, page
    ([1], 0, 1, 1, 1, 64, 16),
    ([0, 1, 15, 16, 17], 0, 1, 4, 4, 128, 16),
    ([63, 64, 65, 300], 0, 1, 8, 2, 128, 32),
    ([777, 3], 0, 1, 2, 1, 256, 64),
    ([5, 0, 40], 1, 1, 8, 8, 64, 16),
    ([100, 33], 130, 1, 8, 2, 128, 64),
    ([2, 257], 513, 1, 4, 2, 256, 32),
    ([5, 7, 0, 200], 100, 5, 4, 4, 64, 16),          # drafts; a sequence shorter than the drafts below
    ([3, 66], 129, 4, 8, 2, 128, 128),
    ([3, 66], 0, 4, 8, 2, 128, 256),                 # rows that see nothing at all
    ([70, 129], 47, 33, 12, 4, 64, 16),              # a chunk
    ([300, 131], 200, 130, 4, 2, 128, 64),
    ([40] * 37, 300, 1, 8, 1, 128, 16),              # many rows behind the prefix
    ([600, 20], 1300, 2, 16, 1, 256, 64),
    ([5000], 0, 1, 4, 1, 128, 16),                   # several ranges
    ([1, 2000], 2900, 3, 2, 2, 64, 32),
    ([200, 150], 0, 40, 4, 2, 64, 16),               # own tokens in the tile kernel: one row tile
    ([513, 400], 65, 100, 4, 1, 128, 32),            # four row tiles, then five
    ([700], 129, 160, 4, 1, 64, 256),
    ([129, 128, 127], 127, 64, 2, 1, 256, 128),
    ([33], 4100, 1, 64, 1, 128, 64),                 # one row tile over a long prefix
    ([5] * 65, 1000, 1, 8, 2, 256, 16),
    ([9000], 0, 1, 2, 1, 64, 16),                    # more than 32 ranges
    ([20000], 0, 2, 1, 1, 128, 64),                  # more than 128 ranges
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])) + "_" + str(len(s[0])))
def test_attention_matches_the_plain_form(shape, fp8):
    p = Problem(*shape, fp8=fp8, seed=7)
    p.check(*p.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", [SHAPES[7], SHAPES[11]], ids=["drafts", "chunk"])
def test_without_the_causal_mask_every_own_key_is_seen(shape, fp8):
    p = Problem(*shape, fp8=fp8, seed=9)
    p.check(*p.run(causal=False), causal=False)


@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_scores_and_a_given_scale(fp8):
    p = Problem([900, 77], 700, 2, 8, 2, 128, 32, fp8, seed=11, kscale=6.0)
    p.check(*p.run(scale=0.25), scale=0.25)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 128])
def test_write_quantises_each_row_exactly(d, ps):
    """Codes and scales, bit for bit: ordinary rows, zeros, one element, the
    smallest subnormals, the largest finite values, padding and a strided source."""
    g = gen(3)
    T, hkv, pages = 203, 3, 203 // ps + 3
    x = rand(g, T, 4 * hkv, d)
    x[0] = 0.0
    x[1, :, 1:] = 0.0
    x[2] = torch.tensor(9.2e-41).to(torch.bfloat16)                  # the smallest bf16
    x[3] = x[3] * 1e-38
    x[4] = torch.finfo(torch.bfloat16).max
    x[5] = x[5] * 1e30
    k, v = x[:, hkv:2 * hkv], x[:, 3 * hkv:]
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T]
    slots[::9] = -1 - torch.arange(len(slots[::9]), device=DEV)
    c = filled_cache(pages, ps, hkv, d, True)
    before = [t.clone() for t in c]
    api.attn_kv_write(k, v, slots, c)
    assert api.device_status()[0] == 0
    kept = slots[slots >= 0]
    page, row = kept // ps, kept % ps
    for n, src, s0, c0 in (("k", k, before[2], before[0]), ("v", v, before[3], before[1])):
        want, scale = ref.quantise(src[slots >= 0])
        assert torch.equal(code_values(getattr(c, n))[page, :, row], want)
        assert torch.equal(getattr(c, n + "_scale")[page, :, row], scale)
        # everything else is as it was
        mask = torch.ones((pages, ps), dtype=torch.bool, device=DEV)
        mask[page, row] = False
        mask = mask[:, None, :].expand(pages, hkv, ps)
        assert torch.equal(getattr(c, n)[mask], c0[mask])
        assert bool(torch.isnan(getattr(c, n + "_scale")[mask]).all())


def test_rows_with_an_infinity_or_a_nan_read_back_as_nan():
    c = api.kv_cache(1, 16, 2, 64)
    x = rand(gen(1), 3, 2, 64)
    x[0, 0, 5] = INF
    x[1, 1, 63] = NAN
    api.attn_kv_write(x, x, torch.arange(3, device=DEV), c)
    k, v = api.attn_kv_read(c, torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                            torch.tensor([3], dtype=torch.int32, device=DEV), 3)
    for t in (k, v):
        nan = torch.isnan(t).all(-1)[0]
        assert nan.tolist() == [[True, False], [False, True], [False, False]]
        assert torch.isfinite(t[0, 2]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,ps,hkv", [(64, 16, 5), (128, 32, 1), (256, 128, 2)])
def test_write_then_read_back(d, ps, hkv, fp8):
    lens = [0, 1, ps - 1, ps, 3 * ps + 5, 40]
    p = Problem(lens, 0, 1, hkv, hkv, d, ps, fp8, seed=4)
    N = 3 * ps + 2                                                     # cuts the longest
    k = torch.full((len(lens), N, hkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    api.attn_kv_read(p.cache, p.table, p.seq_lens, N, out_k=k, out_v=v)
    assert api.device_status()[0] == 0
    for b, n in enumerate(lens):
        n = min(n, N)
        for got, name in ((k, "k"), (v, "v")):
            # code * scale is rounded to float32 (exact in float64) and to bf16
            want = p.values(name, b)[:n].float().to(torch.bfloat16)
            assert torch.equal(got[b, :n], want)
            assert bool((got[b, n:] == 7.0).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_what_a_row_does_not_see_cannot_reach_it(fp8):
    """NaN in the keys and values of the last token: the query tokens before it
    do not notice, the last one does."""
    p = Problem([70, 21], 40, 4, 4, 2, 128, 16, fp8, seed=5)
    o0, l0 = p.run()
    for b, n in enumerate(p.lens):
        slot = int(p.table[b, (n - 1) // 16]) * 16 + (n - 1) % 16
        x = p.k[b + 1][-1:].clone()
        y = p.v[b + 1][-1:].clone()
        y[..., 3] = NAN if b == 0 else INF
        api.attn_kv_write(x, y, torch.tensor([slot], device=DEV), p.cache)
    o1, l1 = p.run()
    assert torch.equal(o1[:, :3], o0[:, :3]) and torch.equal(l1[:, :, :3], l0[:, :, :3])
    assert bool(torch.isnan(o1[:, 3, :, 3]).all())
    for b, n in enumerate(p.lens):
        slot = int(p.table[b, (n - 1) // 16]) * 16 + (n - 1) % 16
        x = torch.full_like(p.k[b + 1][-1:], NAN)
        api.attn_kv_write(x, p.v[b + 1][-1:], torch.tensor([slot], device=DEV), p.cache)
    o2, l2 = p.run()
    assert torch.equal(o2[:, :3], o0[:, :3]) and torch.equal(l2[:, :, :3], l0[:, :, :3])
    assert bool(torch.isnan(o2[:, 3]).all()) and bool(torch.isnan(l2[:, :, 3]).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_what_a_row_of_a_chunk_does_not_see_cannot_reach_it(d, fp8):
    """The same for chunks (tile kernel, one row tile and two): a value row with an
    infinity or a NaN five tokens before the end, then a key row."""
    for Nq, G in ((80, 1), (80, 2)):
        p = Problem([170, 93], 40, Nq, 2 * G, 2, d, 16, fp8, seed=6)
        o0, l0 = p.run()
        free = Nq - 5                      # the queries before it
        for b, n in enumerate(p.lens):
            at = n - 5
            slot = torch.tensor([int(p.table[b, at // 16]) * 16 + at % 16], device=DEV)
            y = p.v[b + 1][at:at + 1].clone()
            y[..., 3] = NAN if b == 0 else -INF
            api.attn_kv_write(p.k[b + 1][at:at + 1], y, slot, p.cache)
        o1, l1 = p.run()
        assert torch.equal(o1[:, :free], o0[:, :free]) and torch.equal(l1[:, :, :free], l0[:, :, :free])
        assert bool(torch.isnan(o1[:, free:]).all()) and bool(torch.isnan(l1[:, :, free:]).all())
        for b, n in enumerate(p.lens):
            at = n - 5
            slot = torch.tensor([int(p.table[b, at // 16]) * 16 + at % 16], device=DEV)
            x = torch.full_like(p.k[b + 1][at:at + 1], NAN)
            api.attn_kv_write(x, p.v[b + 1][at:at + 1], slot, p.cache)
        o2, l2 = p.run()
        assert torch.equal(o2[:, :free], o0[:, :free]) and torch.equal(l2[:, :, :free], l0[:, :, :free])
        assert bool(torch.isnan(o2[:, free:]).all()) and bool(torch.isnan(l2[:, :, free:]).all())
        assert api.device_status()[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_lengths_are_refused_and_reported(fp8):
    """A page outside the cache hides its tokens, a length beyond the table is cut
    to it, a slot beyond the cache is skipped; each is reported once."""
    ps, Nq = 16, 1
    p = Problem([64, 40], 48, Nq, 4, 2, 64, ps, fp8, seed=6)
    pages = p.cache.k.shape[0]
    p.table[0, 1] = pages                   # tokens 16..31 of sequence 0
    p.prefix_table[2] = -1                  # tokens 32..47 of the prefix
    o, lse = p.run()
    rc, site = api.device_status()
    assert rc == -5 and site == 0x102
    assert api.device_status()[0] == 0
    for n in ("k", "v"):
        x = getattr(p, n)
        x[0] = x[0][:32]
        x[1] = torch.cat([x[1][:16], x[1][32:]])
    p.prefix, p.lens = 32, [48, 40]
    p.check(o, lse)
    # lengths: the table has room for max_pages * ps tokens
    p = Problem([64, 40], 0, Nq, 4, 2, 64, ps, fp8, seed=6)
    room = p.table[:, :4].contiguous()
    lens = torch.tensor([1000, 40], dtype=torch.int32, device=DEV)
    o, lse = api.attn_fwd_paged(p.q, p.cache, room, lens)
    assert api.device_status() == (-5, 0x103)
    p.check(o, lse)
    k, v = api.attn_kv_read(p.cache, room, lens, 100)
    assert api.device_status() == (-5, 0x103)
    assert torch.isfinite(k[0, :64]).all() and bool((k[0, 64:] == 0).all())
    # slots
    before = [t.clone() for t in p.cache if t is not None]
    x = rand(gen(2), 2, 2, 64)
    api.attn_kv_write(x, x, torch.tensor([p.cache.k.shape[0] * ps, 1 << 40], device=DEV), p.cache)
    assert api.device_status() == (-5, 0x101)
    for a, b in zip(before, [t for t in p.cache if t is not None]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_strided_block_table_other_stream_and_given_outputs():
    p = Problem([100, 33, 260], 70, 2, 8, 2, 128, 32, True, seed=8)
    full = torch.full((3, 20), -1, dtype=torch.int32, device=DEV)
    full[:, 3:3 + p.table.shape[1]] = p.table
    p.table = full[:, 3:3 + p.table.shape[1]]
    out = torch.empty_like(p.q)
    lse = torch.empty((3, 8, 2), device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, l = p.run(stream=s, out=out, lse=lse)
    s.synchronize()
    assert o is out and l is lse
    p.check(o, l)


def test_decoding_steps_in_a_captured_graph():
    """Write, then attend, captured once and replayed while lengths, slots and
    table entries change; every step equals the eager calls on the same cache."""
    ps, hkv, d, H, B, steps = 16, 2, 128, 8, 3, 20
    p = Problem([10, 1, 31], 50, 1, H, hkv, d, ps, True, seed=12)
    free = torch.arange(p.cache.k.shape[0], device=DEV, dtype=torch.int32)
    table = torch.zeros((B, 5), dtype=torch.int32, device=DEV)
    cache = api.kv_cache(p.cache.k.shape[0] + 15, ps, hkv, d)
    for dst, src in zip(cache, p.cache):
        dst[:src.shape[0]] = src
    own = p.cache.k.shape[0] + torch.arange(15, dtype=torch.int32, device=DEV).view(B, 5)
    for b, n in enumerate(p.lens):
        for x in range(-(-n // ps)):
            for t in cache:
                t[own[b, x]] = t[p.table[b, x]]
    del free
    table.copy_(own)
    g = gen(13)
    lens = p.seq_lens.clone()
    k, v = rand(g, B, hkv, d), rand(g, B, hkv, d)
    q = rand(g, B, 1, H, d)
    slots = torch.zeros(B, dtype=torch.int64, device=DEV)
    ws = torch.empty(api.paged_workspace_bytes(B, 1, H, hkv, d, p.prefix, 5, ps), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((B, H, 1), device=DEV)

    def step():
        api.attn_kv_write(k, v, slots, cache)
        api.attn_fwd_paged(q, cache, table, lens, p.prefix_table, p.prefix, out=out, lse=lse, workspace=ws)

    def place():
        at = lens.long()
        slots.copy_(table.long().gather(1, (at // ps)[:, None])[:, 0] * ps + at % ps)
        lens.add_(1)

    saved = [t.clone() for t in cache]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    place()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens.copy_(p.seq_lens)
    for t, s in zip(cache, saved):
        t.copy_(s)
    for i in range(steps):
        for t in (k, v, q):
            t.copy_(rand(g, *t.shape))
        place()
        graph.replay()
        torch.cuda.synchronize()
        got = (out.clone(), lse.clone())
        step()                                    # the same slots and values again
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i
        for b in range(B):
            p.k[b + 1] = torch.cat([p.k[b + 1], k[b:b + 1]])
            p.v[b + 1] = torch.cat([p.v[b + 1], v[b:b + 1]])
    p.lens = [n + steps for n in p.lens]
    p.q = q
    p.check(out, lse)


def test_a_shared_prefix_equals_the_same_tokens_unshared_and_the_dense_forward():
    """A run of the operators together: a prompt is written, read back and given to
    the dense forward; the paged attention of its last tokens, with a part of it
    as a shared prefix or without, gives the same rows."""
    ps, H, hkv, d, N, Nq = 32, 8, 2, 128, 200, 6
    g = gen(21)
    k, v, q = rand(g, N, hkv, d), rand(g, N, hkv, d), rand(g, 1, N, H, d)
    for fp8 in (False, True):
        cache = filled_cache(9, ps, hkv, d, fp8)
        order = torch.tensor([4, 0, 8, 2, 6, 1, 5], dtype=torch.int32, device=DEV)
        n = torch.arange(N, device=DEV)
        api.attn_kv_write(k, v, order.long()[n // ps] * ps + n % ps, cache)
        table, lens = order[None], torch.tensor([N], dtype=torch.int32, device=DEV)
        kk, vv = api.attn_kv_read(cache, table, lens, N)
        dense, dl = api.attn_fwd(q, kk, vv, causal=True)
        qq = q[:, -Nq:].contiguous()
        alone, al = api.attn_fwd_paged(qq, cache, table, lens)
        both, bl = api.attn_fwd_paged(qq, cache, table[:, 3:], lens - 96, order[:3].contiguous(), 96)
        torch.cuda.synchronize()
        assert api.device_status()[0] == 0
        # each of the two is within its own rounding of the same values
        for o, l in ((alone, al), (both, bl)):
            # bf16 weights and a bf16 result on both sides; the dense side also
            # has K and V rounded to bf16 where the cache is e4m3 (2^-8 on a score
            # of size sum |q k| scale, about 10 here, so 2 * 10 * 2^-8 on a weight)
            tol = 4 * 2.0 ** -8 + (2 * 10 * 2.0 ** -8 if fp8 else 0)
            spread = 1.0
            assert float((o.float() - dense[:, -Nq:].float()).abs().max()) <= tol * spread
            assert float((l - dl[:, :, -Nq:]).abs().max()) <= (10 * 2.0 ** -8 if fp8 else 1e-3)


def test_cache_beyond_32_bit_offsets():
    """Pages past 2^32 bytes (and 2^31 elements) from the start of the cache."""
    ps, hkv, d = 256, 8, 256
    page_bytes = ps * hkv * d
    pages = (1 << 32) // page_bytes + 4
    cache = api.kv_cache(pages, ps, hkv, d)
    g = gen(31)
    N = 300
    k, v, q = rand(g, N, hkv, d), rand(g, N, hkv, d), rand(g, 1, 1, hkv, d)
    order = torch.tensor([pages - 1, pages - 3], dtype=torch.int32, device=DEV)
    n = torch.arange(N, device=DEV)
    api.attn_kv_write(k, v, order.long()[n // ps] * ps + n % ps, cache)
    lens = torch.tensor([N], dtype=torch.int32, device=DEV)
    low = api.kv_cache(2, ps, hkv, d)
    for a, b in zip(low, cache):
        a[0].copy_(b[pages - 1])
        a[1].copy_(b[pages - 3])
    near = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    assert bool((low.k != 0).any())
    for x, y in zip(api.attn_kv_read(cache, order[None], lens, N), api.attn_kv_read(low, near, lens, N)):
        assert torch.equal(x, y) and bool((x[0, N - 1] != 0).any())
    for x, y in zip(api.attn_fwd_paged(q, cache, order[None], lens), api.attn_fwd_paged(q, low, near, lens)):
        assert torch.equal(x, y)
    for x, y in zip(api.attn_fwd_paged(q, cache, order[None], lens * 0, order, N),
                    api.attn_fwd_paged(q, low, near, lens * 0, near[0].contiguous(), N)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Nq", [3, 70])
def test_rows_whose_first_keys_are_masked_or_far_below_the_later_ones(fp8, Nq):
    """Scores of -800 before scores around 0 and the other way round: the running
    reference has to follow, whatever kernel has the rows."""
    p = Problem([300, 260], 400, Nq, 4, 2, 64, 32, fp8, seed=31)
    # q has one large element; the prefix's keys and some own ones oppose it
    p.q[..., 0] = 40.0
    for b, ks in enumerate(p.k):
        ks[..., 0] = 0.0
        n = len(ks)
        if b == 0:
            ks[: n // 2, :, 0] = -160.0
        else:
            ks[n // 3:, :, 0] = -160.0 if b == 1 else 20.0
        t = p.prefix_table if b == 0 else p.table[b - 1]
        i = torch.arange(n, device=DEV)
        api.attn_kv_write(ks, p.v[b], t.long()[i // 32] * 32 + i % 32, p.cache)
    p.check(*p.run())


@pytest.mark.parametrize("Nq", [1, 80])
def test_value_scales_that_differ_by_orders_of_magnitude(Nq):
    """e4m3: the values' row scales ride on the weights, which are kept in 16 bits."""
    p = Problem([400, 90], 700, Nq, 4, 2, 128, 16, True, seed=33)
    g = gen(34)
    for b, vs in enumerate(p.v):
        vs *= torch.exp2(torch.randint(-12, 13, (len(vs), 1, 1), generator=g, device=DEV).float()).to(torch.bfloat16)
        vs[: len(vs) // 4] *= 2.0 ** -40
        t = p.prefix_table if b == 0 else p.table[b - 1]
        i = torch.arange(len(vs), device=DEV)
        api.attn_kv_write(p.k[b], vs, t.long()[i // 16] * 16 + i % 16, p.cache)
    p.check(*p.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Nq", [1, 80])
def test_queries_of_any_magnitude(fp8, Nq):
    """Rows of q from the smallest to the largest bf16 numbers (their scores are
    brought back by the scale), rows of zeros, and one with a NaN."""
    p = Problem([300, 200], 150, Nq, 4, 2, 128, 64, fp8, seed=35)
    p.q[0] *= 2.0 ** 100
    p.q[1] *= 2.0 ** -120
    p.q[0, 0, 1] = 0.0
    o, lse = p.run(scale=2.0 ** -103)
    keep = p.q.clone()
    p.q[1] = 0.0          # 2^-120 2^-103: the scores vanish
    p.check(o, lse, scale=2.0 ** -103)
    p.q.copy_(keep)
    p.q[0, Nq - 1, 2, 77] = NAN
    o2, l2 = p.run(scale=2.0 ** -103)
    bad = torch.isnan(o2).all(-1)
    assert bad.sum() == 1 and bool(bad[0, Nq - 1, 2]) and bool(torch.isnan(l2[0, 2, Nq - 1]))
    o2[0, Nq - 1, 2] = o[0, Nq - 1, 2]
    assert torch.equal(o2, o)


def test_two_calls_at_once_on_two_streams():
    """Each with its own workspace, over one cache; both equal the calls alone."""
    p = Problem([300, 200, 100, 40], 700, 2, 8, 2, 128, 16, True, seed=41)
    r = Problem([600, 31], 300, 40, 8, 2, 128, 16, False, seed=42)
    want = [p.run(), r.run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [x.run(stream=s) for x, s in zip((p, r), streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_calls_in_a_row_share_a_workspace():
    """Ordered on one stream, each overwrites it: shapes that use it differently."""
    ps = [Problem([300, 77], 900, 3, 8, 2, 128, 16, True, seed=14), Problem([50] * 30, 200, 1, 8, 8, 128, 16, False, seed=15),
          Problem([600], 130, 100, 8, 2, 128, 64, True, seed=16)]
    need = max(api.paged_workspace_bytes(x.q.shape[0], x.q.shape[1], 8, x.hkv, 128, x.prefix, x.table.shape[1], x.ps) for x in ps)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    got = [x.run(workspace=ws) for x in ps] + [x.run(workspace=ws) for x in ps]
    for x, g in zip(ps + ps, got):
        x.check(*g)


def test_a_full_reference_of_a_decoding_batch_of_many_sequences():
    p = Problem([(7 * b) % 90 for b in range(200)], 333, 1, 4, 1, 64, 16, True, seed=43)
    p.check(*p.run())


def test_waits_that_run_out_are_reported_and_the_context_survives():
    """A one-cycle limit makes the kernels give up: they return, the host sees the
    status, and the next call is right."""
    lib = api.library()
    for Nq, fp8 in ((1, False), (1, True), (90, False), (90, True)):
        p = Problem([2000, 1500], 2000, Nq, 8, 2, 128, 64, fp8, seed=44)
        want = p.run()
        torch.cuda.synchronize()
        assert api.device_status()[0] == 0
        assert lib.attn_set_wait_limit(1) == 0
        try:
            p.run()
            rc, site = api.device_status()
        finally:
            lib.attn_set_wait_limit(0)
        assert rc in (0, -4)
        if rc:
            assert 0xa1 <= site <= 0xab or site in (0xb1, 0xb2), hex(site)
        assert api.device_status()[0] == 0
        got = p.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert api.device_status()[0] == 0


@pytest.mark.parametrize("change, match", [
    (dict(dtype=torch.float16), "bf16"), (dict(heads=3), "multiple"), (dict(dim=128), "head dim"),
    (dict(table=torch.int64), "block_table"), (dict(lens=torch.int64), "seq_lens"), (dict(short=True), "prefix_table"),
    (dict(flip=True), "contiguous"),
])
def test_binding_refusals(change, match):
    c = api.kv_cache(8, 16, 2, 64)
    q = torch.zeros(2, 1, change.get("heads", 4), change.get("dim", 64), dtype=change.get("dtype", torch.bfloat16), device=DEV)
    if change.get("flip"):
        q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV).expand(2, 4, 2, 64).transpose(1, 2)
    table = torch.zeros(2, 2, dtype=change.get("table", torch.int32), device=DEV)
    lens = torch.ones(2, dtype=change.get("lens", torch.int32), device=DEV)
    pre = torch.zeros(1 if change.get("short") else 4, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match=match):
        api.attn_fwd_paged(q, c, table, lens, pre, 40)


def test_repeated_calls_give_the_same_bits():
    p = Problem([300, 77, 0], 900, 3, 8, 2, 128, 16, True, seed=14)
    o, lse = p.run()
    for _ in range(3):
        o2, l2 = p.run()
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_the_outputs_do_not_depend_on_how_torch_allocates_them(monkeypatch):
    p = Problem([300, 77, 0], 900, 3, 8, 2, 128, 16, True, seed=15)
    o, lse = p.run()
    assert o.is_contiguous() and lse.is_contiguous() and o.dtype == torch.bfloat16 and lse.dtype == torch.float32
    assert o.device == p.q.device and o.shape == p.q.shape and lse.shape == (3, 8, 3)
    for name in ("_raw_empty", "_raw_stream"):
        monkeypatch.setattr(api, name, None)
    o2, l2 = p.run()
    assert o2.stride() == o.stride() and l2.stride() == lse.stride()
    assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_buffers_made_for_another_stream_are_that_streams():
    """Memory freed on the current stream may still be in use there."""
    p = Problem([300, 77, 5], 900, 3, 8, 2, 128, 16, True, seed=16)
    want = p.run()
    need = api.paged_workspace_bytes(3, 3, 8, 2, 128, 900, p.table.shape[1], 16)
    assert need > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(want[0]) for _ in range(8)] + [torch.empty_like(want[1]) for _ in range(8)]
    addresses = {t.data_ptr() for t in freed}
    del freed
    for stream in (side, side.cuda_stream):
        o, lse = p.run(stream=stream)
        assert o.data_ptr() not in addresses and lse.data_ptr() not in addresses
        side.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_empty_problems():
    c = api.kv_cache(2, 16, 2, 64)
    none = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    lens = torch.zeros((0,), dtype=torch.int32, device=DEV)
    api.attn_kv_write(torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV),
                      torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV),
                      torch.zeros((0,), dtype=torch.int64, device=DEV), c)
    k, v = api.attn_kv_read(c, none, lens, 5)
    assert k.shape == (0, 5, 2, 64)
    o, lse = api.attn_fwd_paged(torch.zeros((0, 1, 4, 64), dtype=torch.bfloat16, device=DEV), c, none, lens)
    assert o.shape == (0, 1, 4, 64)
    # no own pages at all and no prefix: rows that see nothing
    q = rand(gen(1), 2, 1, 4, 64)
    o, lse = api.attn_fwd_paged(q, c, torch.zeros((2, 0), dtype=torch.int32, device=DEV),
                                torch.zeros((2,), dtype=torch.int32, device=DEV))
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    assert api.device_status()[0] == 0
