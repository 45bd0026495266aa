"""The paged key/value cache and the attention that reads it: what is measured.

Three operators, on a cache of pages (k and v: (pages, H_kv, page_size, d), in
bf16, or in e4m3 with one float32 scale per row, (pages, H_kv, page_size)):

  write   new tokens' keys and values go to their slots (slot = page *
          page_size + row; negative: the token is padding and is skipped); an
          e4m3 cache quantises each row on the way: scale = amax / 448 (1 for a
          row of zeros), code = e4m3(x / scale)
  read    the first len_b tokens of every sequence back as bf16 (B, N, H_kv,
          d); rows from len_b on are left as they were
  attend  Nq query tokens of each of B sequences against a prefix that all of
          them share (its pages are listed once) followed by each sequence's
          own tokens; the queries are the last Nq of the own tokens

`run` computes them in elementary torch operations where `own` is false, and
through exact_attention_71_gb300.api where it is true.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # One decoding step of 32 sequences: one new token each (latency).
        dict(name="write_step", op="write", T=32, H_kv=8, d=128, page=16, fp8=True, fused=True, pad=0),
        # A prompt of 32768 tokens goes into an e4m3 cache.
        dict(name="write_prompt", op="write", T=32768, H_kv=8, d=128, page=64, fp8=True, fused=False, pad=0),
        # A ragged batch of prompts, head dim 64, cut out of a fused projection, every eleventh token padding.
        dict(name="write_ragged_d64", op="write", T=4999, H_kv=16, d=64, page=16, fp8=True, fused=True, pad=11),
        # Sixteen histories read back for a pass of the dense attention over them.
        dict(name="read_batch", op="read", B=16, N=8192, H_kv=8, d=128, page=64, fp8=True),
        # Three short histories of odd lengths from a bf16 cache of head dim 256.
        dict(name="read_short_d256", op="read", B=3, N=301, H_kv=8, d=256, page=16, fp8=False),
        # A few users behind a short common instruction (latency).
        dict(name="decode_few", op="attend", B=4, Nq=1, H=32, H_kv=8, d=128, prefix=512, own=97, page=16, fp8=True,
             empty=False),
        # One long conversation, nothing shared, multi-head.
        dict(name="decode_one_long", op="attend", B=1, Nq=1, H=16, H_kv=16, d=128, prefix=0, own=16384, page=16,
             fp8=False, empty=False),
        # 64 users behind one long document, grouped heads, e4m3 cache.
        dict(name="decode_shared_e4m3", op="attend", B=64, Nq=1, H=32, H_kv=8, d=128, prefix=8192, own=1024, page=64,
             fp8=True, empty=False),
        # 128 users behind a document of 16384 tokens, bf16 cache: the prefix is a matrix product by now.
        dict(name="decode_shared_bf16", op="attend", B=128, Nq=1, H=32, H_kv=8, d=128, prefix=16384, own=512, page=64,
             fp8=False, empty=False),
        # Five drafted tokens a sequence are verified; odd lengths, head dim 64, one slot of the batch unused.
        dict(name="draft_d64", op="attend", B=24, Nq=5, H=16, H_kv=16, d=64, prefix=4003, own=333, page=16,
             fp8=False, empty=True),
        # Two prompts are processed 512 tokens at a time behind a cached document.
        dict(name="chunk_e4m3", op="attend", B=2, Nq=512, H=32, H_kv=8, d=128, prefix=8192, own=1024, page=64,
             fp8=True, empty=False),
        # Head dim 256, 16 users.
        dict(name="decode_d256", op="attend", B=16, Nq=1, H=8, H_kv=2, d=256, prefix=2048, own=700, page=32,
             fp8=False, empty=False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    while True:
        op = rng.choice(("write", "read", "attend", "attend", "attend"))
        c = dict(op=op, H_kv=rng.choice((1, 2, 4, 8, 16)), d=rng.choice((64, 128, 128, 256)),
                 page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5)
        if op == "write":
            c.update(T=log_int(1, 32768), fused=rng.random() < 0.5, pad=rng.choice((0, 7, 11)))
        elif op == "read":
            c.update(B=log_int(1, 16), N=log_int(1, 8192))
        else:
            Nq = rng.choice((1, 1, 1, 2, 5, 8, log_int(9, 512)))
            c.update(B=log_int(1, 128), Nq=Nq, H=c["H_kv"] * rng.choice((1, 2, 4, 8)),
                     prefix=rng.choice((0, log_int(1, 16384), log_int(1, 16384))), own=Nq + log_int(1, 16384),
                     empty=rng.random() < 0.2)
        w = work(c)
        if w["bytes"] <= 700e6 and w["flops"] <= 160e9:
            return c


def _lens(case):
    """The sequences' lengths: from the case alone."""
    if case["op"] == "read":
        low, high = 0, case["N"]
    else:
        low, high = case["Nq"], case["own"]
    lens = [high - (b * 7919) % ((high - low) // 2 + 1) for b in range(case["B"])]
    if case.get("empty"):
        lens[-1] = 0
    return lens


def work(case):
    d, hkv, es = case["d"], case["H_kv"], 1 if case["fp8"] else 2
    row = 2 * hkv * (d * es + (4 if case["fp8"] else 0))              # a token's keys and values in the cache
    if case["op"] == "write":
        T = sum(not _padding(case, t) for t in range(case["T"]))
        return {"bytes": T * (2 * hkv * d * 2 + row) + 8 * case["T"], "flops": (6 if case["fp8"] else 0) * T * hkv * d}
    lens = _lens(case)
    if case["op"] == "read":
        T = sum(lens)
        return {"bytes": T * (2 * hkv * d * 2 + row) + 4 * case["B"] + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": (2 if case["fp8"] else 0) * T * hkv * d}
    B, Nq, H = case["B"], case["Nq"], case["H"]
    pairs = sum(case["prefix"] * Nq + sum(max(0, n - Nq + 1 + i) for i in range(Nq)) for n in lens)
    tokens = case["prefix"] + sum(lens)
    return {"bytes": tokens * row + B * Nq * H * (4 * d + 4) + 4 * B + 4 * (tokens // case["page"]),
            "flops": 4 * d * H * pairs}


def _padding(case, t):
    return case["pad"] > 0 and t % case["pad"] == case["pad"] - 1


def _quantise(x):
    """Rows of float32 -> (e4m3 codes, float32 scales)."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    page, d, hkv = case["page"], case["d"], case["H_kv"]
    s = dict(case=dict(case))
    if case["op"] == "write":
        T = case["T"]
        pages = -(-T // page) + 3
        s.update(_cache(g, pages, case))
        if case["fused"]:       # k and v are columns of one projection: (T, heads of q, k and v) x d
            x = _rows(g, (T, 4 * hkv, d), False)
            s.update(new_k=x[:, 2 * hkv:3 * hkv], new_v=x[:, 3 * hkv:])
        else:
            s.update(new_k=_rows(g, (T, hkv, d), True), new_v=_rows(g, (T, hkv, d), False))
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = order[t // page] * page + t % page
        if case["pad"]:
            slots = torch.where(t % case["pad"] == case["pad"] - 1, torch.full_like(slots, -1), slots)
        s["slots"] = slots
        return s
    lens = _lens(case)
    per = max(1, -(-max(lens) // page))                                # pages of the longest sequence
    shared = -(-case.get("prefix", 0) // page)
    pages = shared + per * case["B"] + 3
    s.update(_cache(g, pages, case))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["prefix_table"] = order[:shared].clone()
    s["table"] = order[shared:shared + per * case["B"]].view(case["B"], per).clone()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "read":
        shape = (case["B"], case["N"], hkv, d)
        s["out_k"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        s["out_v"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    else:
        s["q"] = _rows(g, (case["B"], case["Nq"], case["H"], d), False)
    return s


def run(s):
    case = s["case"]
    if own:
        from exact_attention_71_gb300 import api
        cache = api.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "write":
            api.attn_kv_write(s["new_k"], s["new_v"], s["slots"], cache)
            return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}
        if case["op"] == "read":
            k, v = api.attn_kv_read(cache, s["table"], s["lens"], case["N"], out_k=s["out_k"], out_v=s["out_v"])
            return dict(k=k, v=v)
        o, lse = api.attn_fwd_paged(s["q"], cache, s["table"], s["lens"], prefix_table=s["prefix_table"],
                                    prefix_len=case["prefix"], causal=True)
        return dict(o=o, lse=lse)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[case["op"]](s)


def _plain_write(s):
    case = s["case"]
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    page, row = slots // case["page"], slots % case["page"]
    k, v = s["new_k"][keep], s["new_v"][keep]
    if not case["fp8"]:
        s["k"][page, :, row] = k
        s["v"][page, :, row] = v
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}
    (k, ks), (v, vs) = _quantise(k.float()), _quantise(v.float())
    s["k"].view(torch.uint8)[page, :, row] = k.view(torch.uint8)
    s["v"].view(torch.uint8)[page, :, row] = v.view(torch.uint8)
    s["k_scale"][page, :, row] = ks
    s["v_scale"][page, :, row] = vs
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


def _plain_read(s):
    N = s["case"]["N"]
    seen = torch.arange(N, device="cuda")[None, :] < s["lens"][:, None]
    for cache, scale, out in ((s["k"], s["k_scale"], s["out_k"]), (s["v"], s["v_scale"], s["out_v"])):
        x = _gather(cache, scale, s["table"])[:, :N].to(torch.bfloat16)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, N - x.shape[1]))
        out.copy_(torch.where(seen[:, :, None, None], x, out))
    return dict(k=s["out_k"], v=s["out_v"])


def _plain_attend(s):
    case = s["case"]
    B, Nq, H, d = s["q"].shape
    hkv, prefix = case["H_kv"], case["prefix"]
    G = H // hkv
    q = s["q"].float().view(B, Nq, hkv, G, d).permute(2, 0, 3, 1, 4)                   # (H_kv, B, G, Nq, d)
    q = q * (1.0 / math.sqrt(d))
    k, v = _gather(s["k"], s["k_scale"], s["table"]), _gather(s["v"], s["v_scale"], s["table"])
    own_k, own_v = k.permute(2, 0, 3, 1), v.permute(2, 0, 1, 3)                        # (H_kv, B, d, L), (.., L, d)
    L = own_k.shape[-1]
    sees = s["lens"][:, None] - Nq + 1 + torch.arange(Nq, device="cuda")[None, :]      # (B, Nq)
    hidden = torch.arange(L, device="cuda")[None, None, :] >= sees[:, :, None]         # (B, Nq, L)
    rows = q.reshape(hkv, B, G * Nq, d)
    own_s = (rows @ own_k).view(hkv, B, G, Nq, L)
    own_s = own_s.masked_fill(hidden[None, :, None], -math.inf)
    k, v = (_gather(s[n], s[n + "_scale"], s["prefix_table"])[:prefix] for n in ("k", "v"))
    pre_k, pre_v = k.permute(1, 2, 0), v.permute(1, 0, 2)                              # (H_kv, d, P), (H_kv, P, d)
    pre_s = (q.reshape(hkv, B * G * Nq, d) @ pre_k).view(hkv, B, G, Nq, prefix)
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
    page = case["page"]

    def values(n):
        x = s[n].float().double()
        return x if s[n + "_scale"] is None else x * s[n + "_scale"].double()[..., None]

    if case["op"] == "write":
        out = {n: (None if s[n] is None else s[n].float().double()) for n in ("k", "v", "k_scale", "v_scale")}
        at = s["slots"].cpu().tolist()
        tok = torch.tensor([t for t, x in enumerate(at) if x >= 0], dtype=torch.long, device="cuda")
        to = s["slots"][tok]
        for n in ("k", "v"):
            x = s["new_" + n][tok].double()
            if case["fp8"]:
                scale = x.abs().max(-1).values / E4M3_MAX
                scale[scale == 0] = 1.0
                out[n + "_scale"][to // page, :, to % page] = scale
                x = _e4m3_64(x / scale[..., None])
            out[n][to // page, :, to % page] = x
        return out
    k, v = values("k"), values("v")
    lens = _lens(case)

    def tokens(x, table, n):
        """n tokens of one sequence: (n, H_kv, d)"""
        x = x[table.long()[: -(-n // page)]]
        return x.permute(0, 2, 1, 3).flatten(0, 1)[:n]

    if case["op"] == "read":
        out = {n: torch.zeros(s["out_k"].shape, dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for b, n in enumerate(lens):
            out["k"][b, :n] = tokens(k, s["table"][b], n)
            out["v"][b, :n] = tokens(v, s["table"][b], n)
        return out
    B, Nq, H, d = s["q"].shape
    group = H // case["H_kv"]
    pre_k = tokens(k, s["prefix_table"], case["prefix"])
    pre_v = tokens(v, s["prefix_table"], case["prefix"])
    o = torch.zeros((B, Nq, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        kb = torch.cat([pre_k, tokens(k, s["table"][b], n)])
        vb = torch.cat([pre_v, tokens(v, s["table"][b], n)])
        if not len(kb):
            continue
        at = torch.arange(len(kb), device="cuda")
        last = case["prefix"] + n - Nq + torch.arange(Nq, device="cuda")               # the last key that a query sees
        mask = (at[None, :] >= case["prefix"]) & (at[None, :] > last[:, None])
        for h in range(case["H_kv"]):
            qh = s["q"][b, :, h * group:(h + 1) * group].double()                      # (Nq, G, d)
            sc = torch.einsum("igd,jd->igj", qh, kb[:, h]) / math.sqrt(d)
            sc = sc.masked_fill(mask[:, None, :], -math.inf)
            z = torch.logsumexp(sc, -1)
            p = torch.exp(sc - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o[b, :, h * group:(h + 1) * group] = torch.einsum("igj,jd->igd", p, vb[:, h])
            lse[b, h * group:(h + 1) * group] = z.transpose(0, 1)
    return dict(o=o, lse=lse)
