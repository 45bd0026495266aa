"""Rotary positions, and a speculative decoding step over the paged cache: what
is measured.

Four operators.  The cache is one of pages (k and v: (pages, H_kv, page_size, d),
in bf16, or in e4m3 with one float32 scale per row):

  rope    rows of q and k are turned by their tokens' positions: pair i of the
          first `rot` elements by row positions[axis[i]] of float32 tables, the
          other elements stay; several axes: time, height and width of an image
          or a video.  inverse: the transposed rotation, the gradient's way back
  append  the same rotation on the way into the cache: q comes back turned, k is
          turned and v taken as it is, both go to their slots (negative: padding,
          nothing is written and q's row becomes 0), quantised for an e4m3 cache
  tree    Nq drafted tokens of each of B sequences, the last Nq of its own tokens,
          are the nodes of a tree (parents: the index of a node's parent, -1: none,
          -2: not a node).  A node sees the shared prefix, the own tokens before the
          drafts, its ancestors and itself
  accept  the accepted path's rows of the cache move up behind the context: token
          len - Nq + j becomes token len - Nq + accepted[j]

`run` computes them in elementary torch operations where `own` is false, and
through exact_attention_71_gb300.api where it is true.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # Training or prefill of text, two sequences of 4096: q and k before the dense attention.
        dict(name="rope_text", op="rope", B=2, N=4096, H=32, H_kv=8, d=128, rot=128, axes=1, mixed=False, inverse=False,
             interleaved=False, fused=False),
        # Gradients of a video model's q and k: three axes in sections, neighbouring pairs, an odd number of tokens.
        dict(name="rope_video_grad", op="rope", B=1, N=7007, H=16, H_kv=16, d=128, rot=128, axes=3, mixed=False,
             inverse=True, interleaved=True, fused=False),
        # One image's patches, head dim 64, rows and columns, half of each head turned; q and k columns of a projection.
        dict(name="rope_image_d64", op="rope", B=1, N=577, H=16, H_kv=16, d=64, rot=32, axes=2, mixed=False,
             inverse=False, interleaved=False, fused=True),
        # One decoding step of 32 sequences (latency).
        dict(name="append_step", op="append", T=32, H=32, H_kv=8, d=128, rot=128, axes=1, mixed=False, interleaved=False,
             page=16, fp8=True, fused=True, pad=0),
        # Prompts of 32768 tokens in all go into an e4m3 cache.
        dict(name="append_prompt", op="append", T=32768, H=32, H_kv=8, d=128, rot=128, axes=1, mixed=False,
             interleaved=False, page=64, fp8=True, fused=False, pad=0),
        # A ragged batch with images: three axes whose pairs alternate, bf16 cache, every eleventh token padding.
        dict(name="append_images_ragged", op="append", T=4999, H=16, H_kv=4, d=128, rot=128, axes=3, mixed=True,
             interleaved=False, page=16, fp8=False, fused=True, pad=11),
        # Eight drafts for each of four users behind a short common instruction (latency).
        dict(name="tree_few", op="tree", B=4, Nq=8, H=32, H_kv=8, d=128, prefix=512, own=97, page=16, fp8=True, width=3,
             empty=False, drop=0),
        # 64 drafts for each of 32 long conversations, bf16 cache.
        dict(name="tree_batch", op="tree", B=32, Nq=64, H=32, H_kv=8, d=128, prefix=0, own=4096, page=64, fp8=False,
             width=12, empty=False, drop=0),
        # 64 users behind one long document, 16 drafts each, some trees smaller, e4m3 cache.
        dict(name="tree_shared_e4m3", op="tree", B=64, Nq=16, H=32, H_kv=8, d=128, prefix=8192, own=1024, page=64,
             fp8=True, width=4, empty=False, drop=3),
        # Head dim 64, multi-head, odd sizes, one slot of the batch unused.
        dict(name="tree_d64_odd", op="tree", B=7, Nq=27, H=16, H_kv=16, d=64, prefix=0, own=2333, page=16, fp8=False,
             width=5, empty=True, drop=0),
        # The accepted paths of 32 trees, e4m3 cache (latency).
        dict(name="accept_step", op="accept", B=32, Nq=64, M=8, H_kv=8, d=128, page=64, own=2048, fp8=True),
        # 512 short trees, bf16 cache, head dim 256.
        dict(name="accept_many_d256", op="accept", B=512, Nq=16, M=5, H_kv=8, d=256, page=16, own=101, fp8=False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    while True:
        op = rng.choice(("rope", "append", "tree", "tree", "accept"))
        d, hkv = rng.choice((64, 128, 128, 256)), rng.choice((1, 2, 4, 8, 16))
        c = dict(op=op, H_kv=hkv, d=d)
        if op in ("rope", "append"):
            axes = rng.choice((1, 1, 2, 3))
            c.update(H=hkv * rng.choice((1, 2, 4, 8)), rot=rng.choice((d, d, d // 2, d - 16)), axes=axes,
                     mixed=axes > 1 and rng.random() < 0.5, interleaved=rng.random() < 0.4, fused=rng.random() < 0.5)
        if op != "rope":
            c.update(page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5)
        if op == "rope":
            c.update(B=rng.choice((1, 2, 3)), N=log_int(1, 8192), inverse=rng.random() < 0.5)
        elif op == "append":
            c.update(T=log_int(1, 32768), pad=rng.choice((0, 7, 11)))
        elif op == "tree":
            Nq = rng.choice((1, 4, 8, 16, log_int(5, 160), log_int(5, 160)))
            c.update(B=log_int(1, 64), Nq=Nq, H=hkv * rng.choice((1, 2, 4, 8)), own=Nq + log_int(1, 8192),
                     prefix=rng.choice((0, log_int(1, 16384))), width=rng.choice((1, 3, max(1, Nq // 5))),
                     drop=rng.choice((0, 0, 3)))
            c["empty"] = c["B"] > 1 and rng.random() < 0.2
        else:
            M = rng.choice((2, 5, 8, 13))
            c.update(B=log_int(1, 512), M=M, Nq=2 * M + log_int(1, 64))
            c["own"] = c["Nq"] + log_int(1, 1024)
            if c["B"] * c["own"] * hkv * d > 1.5e8:        # (the cache that is made for it)
                continue
        w = work(c)
        if w["bytes"] <= 650e6 and w["flops"] <= 90e9:
            return c


def _lens(case):
    """The sequences' own tokens, drafts included: from the case alone."""
    low, high = case["Nq"], case["own"]
    lens = [high - (b * 7919) % ((high - low) // 2 + 1) for b in range(case["B"])]
    if case.get("empty"):
        lens[-1] = 0
    return lens


def _accepted(case):
    """How many drafts of each sequence are accepted: from the case alone."""
    return [1 + (b * 31) % case["M"] for b in range(case["B"])]


def _padding(case, t):
    return case["pad"] > 0 and t % case["pad"] == case["pad"] - 1


def work(case):
    d, hkv = case["d"], case["H_kv"]
    if case["op"] == "rope":
        T = case["B"] * case["N"]
        pos = 8 * case["axes"] * T if case["axes"] > 1 else 0
        return {"bytes": 4 * T * (case["H"] + hkv) * d + 4 * case["N"] * case["rot"] + pos,
                "flops": 3 * T * (case["H"] + hkv) * case["rot"]}
    row = 2 * hkv * (d * (1 if case["fp8"] else 2) + (4 if case["fp8"] else 0))       # a token's keys and values
    if case["op"] == "append":
        T = sum(not _padding(case, t) for t in range(case["T"]))
        return {"bytes": T * (4 * case["H"] * d + 4 * hkv * d + row + 4 * case["rot"] + 8 * case["axes"])
                + (case["T"] - T) * 2 * case["H"] * d + 8 * case["T"],
                "flops": T * (3 * (case["H"] + hkv) * case["rot"] + (6 * hkv * d if case["fp8"] else 0))}
    if case["op"] == "accept":
        moved = sum(n - 1 for n in _accepted(case))         # (the root stays where it is)
        return {"bytes": 2 * moved * row + 4 * case["B"] * (case["M"] + 1) + 8 * moved, "flops": 0}
    B, Nq, H = case["B"], case["Nq"], case["H"]
    lens = _lens(case)
    deep = (case["width"] + 1) / 2                          # a node's parent is so far before it, in the mean
    seen = sum(1 + i / deep for i in range(Nq))             # drafts that the nodes see, about
    nodes = (Nq - Nq // case["drop"]) / Nq if case["drop"] else 1.0
    pairs = sum(nodes * (Nq * (case["prefix"] + max(0, n - Nq)) + (seen if n else 0)) for n in lens)
    tokens = case["prefix"] + sum(lens)
    return {"bytes": tokens * row + B * Nq * H * (4 * d + 4) + 4 * B * (Nq + 1) + 4 * (tokens // case["page"]),
            "flops": 4 * d * H * pairs}


def _quantise(x):
    """Rows of float32 -> (e4m3 codes, float32 scales)."""
    amax = x.abs().amax(-1)
    # (a tensor's division: by a Python number torch multiplies by the reciprocal)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _rows(g, shape, outliers):
    """bf16 rows as a projection gives them: keys have a few channels that stand out."""
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:
        at = torch.randint(0, shape[-1], (3,), generator=g, device="cuda")
        x[..., at] *= 4.0
    return x.to(torch.bfloat16)


def _cache(g, pages, case):
    """A cache whose every row holds something (what earlier users left there)."""
    shape = (pages, case["H_kv"], case["page"], case["d"])
    k, v = _rows(g, shape, True), _rows(g, shape, False)
    if not case["fp8"]:
        return dict(k=k, v=v, k_scale=None, v_scale=None)
    (k, ks), (v, vs) = _quantise(k.float()), _quantise(v.float())
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _pair_axis(case):
    """The axis that each pair turns by: one after the other in sections, or in turn."""
    half, axes = case["rot"] // 2, case["axes"]
    if case["mixed"]:
        return tuple(i % axes for i in range(half))
    return tuple(min(i * axes // half, axes - 1) for i in range(half))


def _positions(g, case, T, limit):
    """int64 (axes, T): one axis: sequences one after the other, from a position of their own; several: pictures of
    25 columns, 23 rows each."""
    t = torch.arange(T, device="cuda")
    if case["axes"] == 1:
        start = torch.randint(0, max(1, limit - T), (1,), generator=g, device="cuda")
        return (t + start)[None].contiguous()
    start = torch.randint(0, limit // 2, (1,), generator=g, device="cuda")
    grid = torch.stack([start + t // 575, start + t // 25 % 23, start + t % 25])
    return (grid if case["axes"] == 3 else grid[1:]).contiguous()


def _tables(rows, rot):
    """Cosines and sines, float32 (rows, rot / 2), of angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, hkv = case["d"], case["H_kv"]
    s = dict(case=dict(case))
    if case["op"] in ("rope", "append"):
        H = case["H"]
        lead = (case["B"], case["N"]) if case["op"] == "rope" else (case["T"],)
        n = lead[-1]
        limit = 2 * n + 1024
        s["cos"], s["sin"] = _tables(n if case["op"] == "rope" and case["axes"] == 1 else limit, case["rot"])
        s["pair_axis"] = _pair_axis(case) if case["axes"] > 1 else None
        if case["fused"]:       # q, k and v are columns of one projection
            x = _rows(g, (*lead, H + 2 * hkv, d), False)
            s.update(q=x[..., :H, :], new_k=x[..., H:H + hkv, :], new_v=x[..., H + hkv:, :])
        else:
            s.update(q=_rows(g, (*lead, H, d), False), new_k=_rows(g, (*lead, hkv, d), True))
            if case["op"] == "append":
                s["new_v"] = _rows(g, (*lead, hkv, d), False)
        if case["op"] == "rope":
            # (a batch of equal layouts shares its positions; text: token n stands at position n)
            s["positions"] = _positions(g, case, n, limit) if case["axes"] > 1 else None
            return s
        page, T = case["page"], case["T"]
        s["positions"] = _positions(g, case, T, limit)
        pages = -(-T // page) + 3
        s.update(_cache(g, pages, case))
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = order[t // page] * page + t % page
        if case["pad"]:
            slots = torch.where(t % case["pad"] == case["pad"] - 1, torch.full_like(slots, -1), slots)
        s["slots"] = slots
        return s
    page, B, Nq = case["page"], case["B"], case["Nq"]
    lens = _lens(case)
    per = max(1, -(-max(lens) // page))                                # pages of the longest sequence
    shared = -(-case.get("prefix", 0) // page)
    pages = shared + per * B + 3
    s.update(_cache(g, pages, case))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["prefix_table"] = order[:shared].clone()
    s["table"] = order[shared:shared + per * B].view(B, per).clone()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "accept":
        # Ascending nodes, the root first; padding behind them.
        M = case["M"]
        nodes = M + torch.rand((B, Nq - M), generator=g, device="cuda").argsort(1)[:, :M - 1].sort(1).values
        nodes = torch.cat([torch.zeros((B, 1), dtype=torch.long, device="cuda"), nodes], 1)
        count = torch.tensor(_accepted(case), device="cuda")
        kept = torch.arange(M, device="cuda")[None, :] < count[:, None]
        s["accepted"] = torch.where(kept, nodes, torch.full_like(nodes, -1)).to(torch.int32)
        return s
    s["q"] = _rows(g, (B, Nq, case["H"], d), False)
    # A node's parent is one of the `width` nodes before it; the first ones may have none.
    i = torch.arange(Nq, device="cuda")
    back = 1 + (torch.rand((B, Nq), generator=g, device="cuda") * case["width"]).long().clamp(max=case["width"] - 1)
    parents = (i[None, :] - back).clamp(min=-1)
    if case["drop"]:            # smaller trees: the last nodes are none
        parents[:, Nq - Nq // case["drop"]:] = -2
    s["parents"] = parents.to(torch.int32)
    return s


def run(s):
    case = s["case"]
    if own:
        from exact_attention_71_gb300 import api
        if case["op"] == "rope":
            q, k = api.attn_rope(s["q"], s["new_k"], s["cos"], s["sin"], positions=s["positions"],
                                 pair_axis=s["pair_axis"], interleaved=case["interleaved"], inverse=case["inverse"])
            return dict(q=q, k=k)
        cache = api.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "append":
            q = api.attn_kv_append(s["q"], s["new_k"], s["new_v"], s["positions"] if case["axes"] > 1 else s["positions"][0],
                                   s["slots"], cache, s["cos"], s["sin"], pair_axis=s["pair_axis"],
                                   interleaved=case["interleaved"])
            return dict(q=q, **{n: s[n] for n in ("k", "v", "k_scale", "v_scale")})
        if case["op"] == "accept":
            api.attn_kv_accept(cache, s["table"], s["lens"], s["accepted"], case["Nq"])
            return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}
        o, lse = api.attn_fwd_paged_tree(s["q"], cache, s["table"], s["lens"], s["parents"],
                                         prefix_table=s["prefix_table"], prefix_len=case["prefix"])
        return dict(o=o, lse=lse)
    return {"rope": _plain_rope, "append": _plain_append, "tree": _plain_tree, "accept": _plain_accept}[case["op"]](s)


def _turn(x, s, sign):
    """Rows (.., T, heads, d) turned by their tokens' positions, in float32."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    n = x.shape[-3]
    if s["positions"] is None:
        c, sn = s["cos"][:n], s["sin"][:n]
    else:
        axis = torch.tensor(s["pair_axis"] or (0,) * half, device="cuda")
        at = s["positions"][axis].T                                                    # (T, half): the row of each pair
        c, sn = s["cos"].gather(0, at), s["sin"].gather(0, at)
    c, sn = c[:, None, :], sn[:, None, :] * sign
    x = x.float()
    turned, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * c - b * sn, a * sn + b * c], -1)
    return torch.cat([turned, rest], -1)


def _plain_rope(s):
    sign = -1.0 if s["case"]["inverse"] else 1.0
    return dict(q=_turn(s["q"], s, sign).to(torch.bfloat16), k=_turn(s["new_k"], s, sign).to(torch.bfloat16))


def _plain_append(s):
    case = s["case"]
    keep = s["slots"] >= 0
    q = torch.where(keep[:, None, None], _turn(s["q"], s, 1.0), 0.0).to(torch.bfloat16)
    slots = s["slots"][keep]
    page, row = slots // case["page"], slots % case["page"]
    k, v = _turn(s["new_k"], s, 1.0)[keep], s["new_v"][keep].float()
    if not case["fp8"]:
        s["k"][page, :, row] = k.to(torch.bfloat16)
        s["v"][page, :, row] = v.to(torch.bfloat16)
    else:
        (k, ks), (v, vs) = _quantise(k), _quantise(v)
        s["k"].view(torch.uint8)[page, :, row] = k.view(torch.uint8)
        s["v"].view(torch.uint8)[page, :, row] = v.view(torch.uint8)
        s["k_scale"][page, :, row] = ks
        s["v_scale"][page, :, row] = vs
    return dict(q=q, **{n: s[n] for n in ("k", "v", "k_scale", "v_scale")})


def _plain_accept(s):
    page = s["case"]["page"]
    at = s["accepted"].long()
    kept = at >= 0
    start = (s["lens"].long() - s["case"]["Nq"])[:, None]
    here, there = start + torch.where(kept, at, 0), start + torch.arange(at.shape[1], device="cuda")[None, :]
    source, target = s["table"].long().gather(1, here // page)[kept], s["table"].long().gather(1, there // page)[kept]
    here, there = (here % page)[kept], (there % page)[kept]
    for n in ("k", "v", "k_scale", "v_scale"):
        if s[n] is not None:
            x = s[n].view(torch.uint8) if s[n].dtype == torch.float8_e4m3fn else s[n]
            x[target, :, there] = x[source, :, here]
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}


def _gather(cache, scale, table):
    """The tokens of the pages in `table` (..., P), as float32 (..., P * page, H_kv, d)."""
    table = table.long()
    if scale is None:
        x = cache[table].float()
    else:
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scale[table][..., None]
    x = x.transpose(-3, -2)                                            # (..., P, page, H_kv, d)
    return x.reshape(*table.shape[:-1], -1, *x.shape[-2:])


def _plain_tree(s):
    case = s["case"]
    B, Nq, H, d = s["q"].shape
    hkv, prefix = case["H_kv"], case["prefix"]
    G = H // hkv
    parents = s["parents"].long()
    node = parents > -2                                                                # (B, Nq)
    # reach[b, i, j]: j is i or an ancestor of i; paths of 1, 2, 4, .. steps
    j = torch.arange(Nq, device="cuda")
    reach = (parents[:, :, None] == j) | (j[:, None] == j)
    for _ in range(max(1, (Nq - 1).bit_length())):
        reach = (reach.float() @ reach.float()) > 0
    q = s["q"].float().view(B, Nq, hkv, G, d).permute(2, 0, 3, 1, 4)                   # (H_kv, B, G, Nq, d)
    q = q * (1.0 / math.sqrt(d))
    k, v = _gather(s["k"], s["k_scale"], s["table"]), _gather(s["v"], s["v_scale"], s["table"])
    own_k, own_v = k.permute(2, 0, 3, 1), v.permute(2, 0, 1, 3)                        # (H_kv, B, d, L), (.., L, d)
    L = own_k.shape[-1]
    at = torch.arange(L, device="cuda")[None, :] - (s["lens"].long() - Nq)[:, None]    # a key's node: < 0 before the drafts
    drafts = reach.gather(2, at.clamp(0, Nq - 1)[:, None, :].expand(B, Nq, L))
    sees = torch.where(at[:, None, :] < 0, torch.ones_like(drafts), drafts & (at < Nq)[:, None, :])
    hidden = ~(sees & node[:, :, None])
    rows = q.reshape(hkv, B, G * Nq, d)
    own_s = (rows @ own_k).view(hkv, B, G, Nq, L)
    own_s = own_s.masked_fill(hidden[None, :, None], -math.inf)
    k, v = (_gather(s[n], s[n + "_scale"], s["prefix_table"])[:prefix] for n in ("k", "v"))
    pre_k, pre_v = k.permute(1, 2, 0), v.permute(1, 0, 2)                              # (H_kv, d, P), (H_kv, P, d)
    pre_s = (q.reshape(hkv, B * G * Nq, d) @ pre_k).view(hkv, B, G, Nq, prefix)
    pre_s = pre_s.masked_fill(~node[None, :, None, :, None], -math.inf)
    top = own_s.amax(-1)
    if prefix:
        top = torch.maximum(top, pre_s.amax(-1))
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    own_p, pre_p = torch.exp(own_s - top[..., None]), torch.exp(pre_s - top[..., None])
    total = own_p.sum(-1) + pre_p.sum(-1)
    o = (own_p.reshape(hkv, B, G * Nq, L) @ own_v).view(*total.shape, d)
    o = o + (pre_p.reshape(hkv, B * G * Nq, prefix) @ pre_v).view(*total.shape, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    lse = top + torch.log(total)
    return dict(o=o.permute(1, 3, 0, 2, 4).reshape(B, Nq, H, d).to(torch.bfloat16),
                lse=lse.permute(1, 0, 2, 3).reshape(B, H, Nq))


def _e4m3_64(y):
    """float64 -> the nearest e4m3 value (ties to even), saturating at 448."""
    a = y.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    page, d = case.get("page"), case["d"]

    def turned(x, sign):
        """Rows (T, heads, d) in 64 bits: every pair is a complex number that is turned by another."""
        half = case["rot"] // 2
        pos = s["positions"]
        unit = torch.complex(s["cos"].double(), sign * s["sin"].double())
        if pos is None:
            by = unit[torch.arange(x.shape[0], device="cuda")]
        else:
            by = torch.stack([unit[pos[s["pair_axis"][i] if s["pair_axis"] else 0], i] for i in range(half)], -1)
        y = x.double().clone()
        at = torch.arange(half, device="cuda")
        first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
        z = torch.complex(y[..., first], y[..., second]) * by[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if case["op"] == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return {o: torch.stack([turned(x, sign) for x in s[n]]) for o, n in (("q", "q"), ("k", "new_k"))}
    if case["op"] in ("append", "accept"):
        out = {n: (None if s[n] is None else s[n].float().double()) for n in ("k", "v", "k_scale", "v_scale")}
    if case["op"] == "accept":
        before = {n: (None if x is None else x.clone()) for n, x in out.items()}
        table, lens, accepted = s["table"].cpu(), s["lens"].cpu(), s["accepted"].cpu()
        frm, to = [], []
        for b in range(case["B"]):
            start = int(lens[b]) - case["Nq"]
            for j in range(case["M"]):
                if accepted[b, j] >= 0:
                    for rows, tok in ((frm, start + int(accepted[b, j])), (to, start + j)):
                        rows.append((int(table[b, tok // page]), tok % page))
        frm, to = torch.tensor(frm, device="cuda").T, torch.tensor(to, device="cuda").T
        for n, x in out.items():
            if x is not None:
                x[to[0], :, to[1]] = before[n][frm[0], :, frm[1]]
        return out
    if case["op"] == "append":
        tok = torch.nonzero(s["slots"] >= 0)[:, 0]
        to = s["slots"][tok]
        q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        q[tok] = turned(s["q"], 1.0)[tok]
        for n, x in (("k", turned(s["new_k"], 1.0)[tok]), ("v", s["new_v"][tok].double())):
            if case["fp8"]:
                scale = x.abs().max(-1).values / E4M3_MAX
                scale[scale == 0] = 1.0
                out[n + "_scale"][to // page, :, to % page] = scale
                x = _e4m3_64(x / scale[..., None])
            out[n][to // page, :, to % page] = x
        return dict(q=q, **out)

    def values(n):
        x = s[n].float().double()
        return x if s[n + "_scale"] is None else x * s[n + "_scale"].double()[..., None]

    def tokens(x, table, n):
        """n tokens of one sequence: (n, H_kv, d)"""
        x = x[table.long()[: -(-n // page)]]
        return x.permute(0, 2, 1, 3).flatten(0, 1)[:n]

    k, v = values("k"), values("v")
    lens, parents = _lens(case), s["parents"].cpu().tolist()
    B, Nq, H, _ = s["q"].shape
    group = H // case["H_kv"]
    pre_k = tokens(k, s["prefix_table"], case["prefix"])
    pre_v = tokens(v, s["prefix_table"], case["prefix"])
    o = torch.zeros((B, Nq, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        kb = torch.cat([pre_k, tokens(k, s["table"][b], n)])
        vb = torch.cat([pre_v, tokens(v, s["table"][b], n)])
        first = len(kb) - min(n, Nq)                                   # the first key that is a draft
        mask = torch.ones((Nq, len(kb)), dtype=torch.bool)             # hidden
        for i in range(Nq):
            if parents[b][i] < -1 or not len(kb):
                continue
            mask[i, :first] = False
            at = i
            while at >= 0:
                if n >= Nq:
                    mask[i, first + at] = False
                at = parents[b][at]
        mask = mask.cuda()
        if not len(kb):
            continue
        for h in range(case["H_kv"]):
            qh = s["q"][b, :, h * group:(h + 1) * group].double()                      # (Nq, G, d)
            sc = torch.einsum("igd,jd->igj", qh, kb[:, h]) / math.sqrt(d)
            sc = sc.masked_fill(mask[:, None, :], -math.inf)
            z = torch.logsumexp(sc, -1)
            p = torch.exp(sc - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o[b, :, h * group:(h + 1) * group] = torch.einsum("igj,jd->igd", p, vb[:, h])
            lse[b, h * group:(h + 1) * group] = z.transpose(0, 1)
    return dict(o=o, lse=lse)
