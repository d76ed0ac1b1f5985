"""The paged cache's rotating append, the block-scaled e4m3 cache's attention and its block summaries: the cases that are
measured, their plain forms, and the library's calls for them.

A cache of kind ``fp8_block`` holds e4m3 codes and one power-of-two scale per page (a page is one kv head's block).
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE_EXP = -117  # the scale of a block that holds only zeros
CODE = torch.float8_e4m3fn
DEV = "cuda"


def _append(name, kind, batch, hq, hkv, d, block, ctx_min, ctx_max, new_min, new_max, rotary, interleaved, summaries):
    c = {"op": "append", "kind": kind, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max, "new_min": new_min, "new_max": new_max, "rotary": rotary, "interleaved": interleaved,
         "summaries": summaries}
    return dict(c, name=name) if name else c


def _attend(name, batch, hq, hkv, d, block, ctx_min, ctx_max, keep):
    c = {"op": "attend", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max, "keep": keep}
    return dict(c, name=name) if name else c


def _summaries(name, batch, hq, hkv, d, block, ctx_min, ctx_max):
    c = {"op": "summaries", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token of one request: the smallest call, its latency counts
        _append("append_token_b1", "fp8_block", 1, 32, 4, 128, 64, 1000, 1000, 1, 1, 128, False, True),
        # one token each of a full decode batch with requests of very different lengths, 16-token pages
        _append("append_tokens_b256_bf16", "bf16", 256, 32, 4, 128, 16, 500, 9000, 1, 1, 128, False, True),
        # a chunk of one long prompt that ends inside a block and starts inside another
        _append("append_chunk_2000", "fp8_block", 1, 32, 8, 128, 64, 5003, 5003, 2000, 2000, 128, False, True),
        # small fp32 cache, a quarter of each head rotated in neighbouring pairs, odd lengths, some requests with no new token
        _append("append_ragged_f32", "f32", 5, 8, 2, 64, 16, 0, 700, 0, 333, 16, True, True),
        # prompts of a whole batch into the block-scaled cache: the largest
        _append("append_prompts_16x4k", "fp8_block", 16, 32, 4, 128, 64, 0, 130, 1000, 4096, 128, False, True),
        # one short request over its whole cache
        _attend("attend_b1_500", 1, 32, 4, 128, 64, 500, 500, 0),
        # a decode batch over the selected 64 blocks of 131072-token requests (budget of 4096 tokens)
        _attend("attend_selected_b32", 32, 32, 4, 128, 64, 20000, 131072, 64),
        # a batch of uneven requests over their whole caches, 16-token pages
        _attend("attend_ragged_b24", 24, 16, 4, 128, 16, 37, 20011, 0),
        # 16 query heads to a kv head, 64 channels
        _attend("attend_g16_d64", 12, 32, 2, 64, 32, 3001, 40000, 0),
        # the largest: long requests over their whole caches
        _attend("attend_b16_131072", 16, 32, 4, 128, 64, 131072, 131072, 0),
        # summaries of a few short requests, and of a batch of long uneven ones with 16-token pages
        _summaries("summaries_b2_2500", 2, 32, 4, 128, 64, 1200, 2500),
        _summaries("summaries_b32_64k", 32, 32, 4, 128, 16, 4096, 65536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "summaries"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8, 8, 16])
    while hq > 32:
        hq //= 2
    block = rng.choice([16, 32, 64, 128, 16, 64, 48])
    batch = _log(rng, 1, 64)
    if op == "append":
        kind = rng.choice(["fp8_block", "fp8_block", "bf16", "fp8", "f32"])
        rotary = rng.choice([d, d, d // 2, 16])
        ctx = _log(rng, 1, 12000)
        if rng.random() < 0.4:
            return _append(None, kind, batch, hq, hkv, d, block, rng.randrange(ctx), ctx, 1, 1, rotary,
                           rng.random() < 0.3, rng.random() < 0.8)
        new = _log(rng, 2, max(2, 32000 // batch))
        return _append(None, kind, batch, hq, hkv, d, block, 0, min(ctx, 4000), rng.randrange(new), new, rotary,
                       rng.random() < 0.3, rng.random() < 0.8)
    most = min(131072, 8000000 // (hkv * d // 64) // batch // 2)
    ctx = _log(rng, 1, most)
    low = rng.randrange(max(1, ctx // 10), ctx + 1)
    if op == "attend":
        return _attend(None, batch, hq, hkv, d, block, low, ctx, rng.choice([0, 0, 8, 33, 64]))
    return _summaries(None, batch, hq, hkv, d, block, low, ctx)


# ---- what a case is, by its fields alone ---------------------------------------------------------------------------------


def _lens(case, lo, hi, salt):
    """One length per request in [lo, hi], the largest among them."""
    r = random.Random("%s %d %d %d" % (salt, case["batch"], lo, hi))
    got = [r.randint(lo, hi) for _ in range(case["batch"])]
    got[r.randrange(len(got))] = hi
    return got


def _new(case):
    return _lens(case, case["new_min"], case["new_max"], "new")


def _seq_lens(case):
    """Tokens of each request, its new ones included."""
    ctx = _lens(case, case["ctx_min"], case["ctx_max"], "ctx")
    return [c + n for c, n in zip(ctx, _new(case))] if case["op"] == "append" else ctx


def _blocks(case):
    return [-(-n // case["block"]) for n in _seq_lens(case)]


def _touched(case):
    """Blocks that get new tokens."""
    b = case["block"]
    return sum(-(-L // b) - (L - n) // b for L, n in zip(_seq_lens(case), _new(case)) if n)


def _pad_rows(case):
    """Rows behind the last request's: a padded batch."""
    return 0 if case["new_max"] == 1 else 5


def _attended(case):
    """Tokens of each request that its query reads (the kept blocks include the newest)."""
    return [L if not case["keep"] or -(-L // case["block"]) <= case["keep"]
            else (case["keep"] - 1) * case["block"] + (L - 1) % case["block"] + 1 for L in _seq_lens(case)]


def work(case):
    hq, hkv, d, batch = case["hq"], case["hkv"], case["d"], case["batch"]
    if case["op"] == "append":
        src = 4 if case["kind"] == "f32" else 2
        held = {"f32": 4.0, "bf16": 2.0, "fp8": 1.125, "fp8_block": 1.0}[case["kind"]]
        rows = sum(_new(case))
        b = rows * ((2 * hq + 2 * hkv) * d * src + 2 * hkv * d * held + case["rotary"] * 4) + 8 * batch
        if case["summaries"]:
            b += _touched(case) * hkv * 2 * d * src
        return {"bytes": b, "flops": rows * (hq + hkv) * case["rotary"] * 3}
    if case["op"] == "attend":
        tokens = sum(_attended(case))
        sel = sum(-(-n // case["block"]) for n in _attended(case))
        return {"bytes": tokens * hkv * 2 * d + sel * hkv * 16 + batch * hq * (4 * d + 4), "flops": tokens * hq * d * 4}
    blocks = sum(_blocks(case))
    return {"bytes": hkv * (sum(_seq_lens(case)) * d + blocks * (4 * d + 8)), "flops": sum(_seq_lens(case)) * hkv * d * 2}


# ---- inputs --------------------------------------------------------------------------------------------------------------


def _values(shape, g, heavy):
    """N(0, 1.3) rows, a few of them (the heavy ones) larger."""
    x = torch.randn(shape, generator=g, device=DEV) * 1.3
    if heavy:
        x *= 1 + 1.1 * (torch.rand(shape[:-1] + (1,), generator=g, device=DEV) < 0.02)
    return x


def _pool(case, g):
    """Page table of every request's blocks over a shuffled pool with spare pages."""
    blocks, hkv = _blocks(case), case["hkv"]
    mb = max(1, max(blocks))
    used = sum(blocks) * hkv
    pages = used + 3
    order = torch.randperm(pages, generator=g, device=DEV)[:used].to(torch.int32)
    nb = torch.tensor(blocks, device=DEV)
    there = (torch.arange(mb, device=DEV)[None, None, :] < nb[:, None, None]).expand(case["batch"], hkv, mb)
    table = torch.full((case["batch"], hkv, mb), -1, dtype=torch.int32, device=DEV)
    table[there] = order
    return table, pages


def _cache(case, kind, g):
    """Pages with values in them, and the scales that go with the codes."""
    table, pages = _pool(case, g)
    shape = (pages, case["block"], case["d"])
    s = {"table": table, "k_scales": None, "v_scales": None}
    for w in ("k", "v"):
        if kind == "f32":
            s[w] = _values(shape, g, w == "k")
        elif kind == "bf16":
            s[w] = _values(shape, g, w == "k").to(torch.bfloat16)
        elif kind == "fp8":
            s[w] = (torch.randn(shape, generator=g, device=DEV) * 120).clamp(-E4M3_MAX, E4M3_MAX).to(CODE)
            s[w + "_scales"] = 0.004 + 0.012 * torch.rand(shape[:2] + (case["d"] // 32,), generator=g, device=DEV)
        else:
            s[w] = (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(CODE)
            s[w + "_scales"] = torch.exp2(torch.randint(-8, -5, (pages,), generator=g, device=DEV).float())
    return s


def _held(s, kind, w):
    """What the pages stand for, in 32 bits."""
    x = s[w].float()
    if kind == "fp8":
        return x * s[w + "_scales"].repeat_interleave(32, -1)
    return x * s[w + "_scales"][:, None, None] if kind == "fp8_block" else x


def _outward(lo, hi):
    """bf16 bounds at or below lo, at or above hi (finite values)."""
    def down(x):
        y = x.to(torch.bfloat16)
        return torch.where(y.double() > x.double(), torch.nextafter(y, torch.full_like(y, -math.inf)), y)
    return down(lo), -down(-hi)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    batch, hq, hkv, d, block = case["batch"], case["hq"], case["hkv"], case["d"], case["block"]
    kind = case.get("kind", "fp8_block")
    s = {"case": dict(case), "kind": kind}
    s.update(_cache(case, kind, g))
    seq = _seq_lens(case)
    s["seq_lens"] = torch.tensor(seq, dtype=torch.int32, device=DEV)
    mb = s["table"].shape[2]
    if case["op"] == "append":
        new = _new(case)
        wide = torch.float32 if kind == "f32" else torch.bfloat16
        rows = sum(new) + _pad_rows(case)
        # the rows of a fused projection: q, k and v are views of it
        qkv = _values((rows, hq + 2 * hkv, d), g, True).to(wide)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.zeros((rows, hq, d), dtype=wide, device=DEV)
        one = case["new_min"] == case["new_max"] == 1
        s["offsets"] = None if one else torch.tensor([sum(new[:i]) for i in range(batch + 1)], dtype=torch.int32, device=DEV)
        h = case["rotary"] // 2
        inv = 10000.0 ** (-torch.arange(h, device=DEV, dtype=torch.float64) / h)
        angle = torch.arange(max(1, max(seq)), device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["smin"] = s["smax"] = None
        if case["summaries"]:  # of what the cache holds before the new tokens
            dt = torch.float32 if kind == "f32" else torch.bfloat16
            s["smin"] = torch.zeros((batch, hkv, mb, d), dtype=dt, device=DEV)
            s["smax"] = torch.zeros_like(s["smin"])
            old = torch.tensor([L - n for L, n in zip(seq, new)], device=DEV)
            lo, hi = _page_summaries(s, kind, old)
            s["smin"].copy_(lo)
            s["smax"].copy_(hi)
    elif case["op"] == "attend":
        s["q"] = (torch.randn((batch, hq, d), generator=g, device=DEV)).to(torch.bfloat16)
        keep, nb = case["keep"], _blocks(case)
        cap = min(max(nb), keep) if keep else max(nb)
        # the newest block and others at random, ascending
        nbt = torch.tensor(nb, device=DEV)
        j = torch.arange(mb, device=DEV)
        rank = torch.rand((batch, hkv, mb), generator=g, device=DEV) + 2.0 * (j[None, None] == nbt[:, None, None] - 1)
        rank.masked_fill_(j[None, None] >= nbt[:, None, None], -1.0)
        top, at = rank.topk(cap, -1)
        at = torch.where(top >= 0, at, mb).sort(-1).values
        s["sel"] = torch.where(at < mb, at, -1).to(torch.int32).contiguous()
        s["sel_count"] = (s["sel"] >= 0).sum(-1).to(torch.int32).contiguous()
        s["out"] = torch.empty((batch, hq, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((batch, hq), dtype=torch.float32, device=DEV)
    else:
        s["smin"] = torch.zeros((batch, hkv, mb, d), dtype=torch.bfloat16, device=DEV)
        s["smax"] = torch.zeros_like(s["smin"])
    if own:  # the descriptors and the workspace that a program keeps from step to step
        _describe(s)
    return s


# ---- plain forms ---------------------------------------------------------------------------------------------------------


def _page_summaries(s, kind, lens):
    """min / max over the first `lens` tokens of every request, by block; 0 where a block has none."""
    table = s["table"].long()
    batch, hkv, mb = table.shape
    block, d = s["k"].shape[1:]
    valid = (lens[:, None, None] - torch.arange(mb, device=DEV) * block).clamp(0, block).expand(batch, hkv, mb)
    there = valid > 0
    count = torch.zeros(s["k"].shape[0], dtype=torch.long, device=DEV)
    count[table[there]] = valid[there]
    gone = torch.arange(block, device=DEV)[None, :, None] >= count[:, None, None]
    x = s["k"].float() if kind in ("fp8_block",) else _held(s, kind, "k")
    lo, hi = x.masked_fill(gone, math.inf).amin(1), x.masked_fill_(gone, -math.inf).amax(1)
    if kind == "fp8_block":
        lo, hi = lo * s["k_scales"][:, None], hi * s["k_scales"][:, None]
    if kind != "f32":
        lo, hi = _outward(lo, hi)
    zero = torch.zeros((), dtype=lo.dtype, device=DEV)
    at = table.clamp(min=0)
    return (torch.where(there[..., None], lo[at], zero), torch.where(there[..., None], hi[at], zero))


def _rotate(x, cos, sin, rotary, interleaved):
    h = rotary // 2
    r, rest = x[..., :rotary], x[..., rotary:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :h], r[..., h:])
    c, s = cos[:, None], sin[:, None]
    u, v = a * c - b * s, b * c + a * s
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1)


def _rows(s):
    """Request, cache position and whether it is one, of every row."""
    rows, batch = s["q"].shape[0], s["table"].shape[0]
    at = torch.arange(rows, device=DEV)
    offsets = s["offsets"].long() if s["offsets"] is not None else torch.arange(batch + 1, device=DEV)
    req = torch.bucketize(at, offsets[1:].contiguous(), right=True)
    real = req < batch
    req = req.clamp(max=batch - 1)
    pos = s["seq_lens"].long()[req] - offsets[req + 1] + at
    return req, pos, real


def _scale_for(amax):
    """The smallest power of two that amax / 448 does not pass."""
    m, e = torch.frexp(amax / E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=MIN_SCALE_EXP)
    e = torch.where(amax > 0, e, MIN_SCALE_EXP)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _append_plain(s):
    case, kind = s["case"], s["kind"]
    rotary, inter, block = case["rotary"], case["interleaved"], case["block"]
    req, pos, real = _rows(s)
    wide = torch.float64 if kind.startswith("fp8") else torch.float32  # codes: values next to a border
    cos, sin = s["cos_sin"][pos.clamp(0, len(s["cos_sin"]) - 1)].split(rotary // 2, 1)
    q = _rotate(s["q"].float(), cos, sin, rotary, inter).to(s["q_out"].dtype)
    s["q_out"].copy_(torch.where(real[:, None, None], q, s["q_out"]))
    req, pos = req[real], pos[real]
    j, r = pos // block, pos % block
    pages = s["table"].long()[req, :, j]  # [rows, hkv]
    new = {"k": _rotate(s["k_new"].to(wide), cos.to(wide), sin.to(wide), rotary, inter)[real], "v": s["v_new"].to(wide)[real]}
    old = torch.zeros(s["k"].shape[0], dtype=torch.long, device=DEV)  # rows that a touched page held before
    first = torch.full_like(old, block)
    first.scatter_reduce_(0, pages.flatten(), r[:, None].expand_as(pages).flatten(), "amin")
    old = torch.where(first < block, first, old)
    for w in ("k", "v"):
        x = new[w]
        if kind == "fp8_block":
            scales = s[w + "_scales"]
            amax = torch.zeros(scales.shape, dtype=wide, device=DEV)
            amax.scatter_reduce_(0, pages.flatten(), x.abs().amax(-1).flatten(), "amax")
            touched = first < block
            want = _scale_for(amax)
            now = torch.where(touched, torch.where(first > 0, torch.maximum(scales, want), want), scales)
            grown = (touched & (first > 0) & (now > scales)).nonzero()[:, 0]
            again = (s[w][grown].float() * (scales / now)[grown, None, None]).to(CODE)
            keep = torch.arange(block, device=DEV)[None, :, None] < first[grown, None, None]
            s[w].view(torch.uint8)[grown] = torch.where(keep, again.view(torch.uint8), s[w].view(torch.uint8)[grown])
            scales.copy_(now)
            codes = (x / now[pages][..., None].to(wide)).clamp(-E4M3_MAX, E4M3_MAX).float().to(CODE)
            s[w].view(torch.uint8)[pages, r[:, None]] = codes.view(torch.uint8)
        elif kind == "fp8":
            group = x.unflatten(-1, (-1, 32))
            amax = group.abs().amax(-1).float()
            scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
            codes = (group / scale[..., None].to(wide)).clamp(-E4M3_MAX, E4M3_MAX).float().to(CODE).flatten(-2)
            s[w].view(torch.uint8)[pages, r[:, None]] = codes.view(torch.uint8)
            s[w + "_scales"][pages, r[:, None]] = scale
        else:
            s[w][pages, r[:, None]] = x.to(s[w].dtype)
    if s["smin"] is not None:
        lo, hi = _page_summaries(s, kind, s["seq_lens"].long())
        mb = s["table"].shape[2]
        n = torch.bincount(req, minlength=s["table"].shape[0])
        start = (s["seq_lens"].long() - n) // block
        cols = torch.arange(mb, device=DEV)[None]
        mine = ((n > 0)[:, None] & (cols >= start[:, None]) & (cols * block < s["seq_lens"][:, None]))[:, None, :, None]
        s["smin"].copy_(torch.where(mine, lo, s["smin"]))
        s["smax"].copy_(torch.where(mine, hi, s["smax"]))
    return _append_out(s)


def _append_out(s):
    return {k: s[k] for k in ("q_out", "k", "v", "k_scales", "v_scales", "smin", "smax")}


def _attend_plain(s):
    case = s["case"]
    batch, hkv, d, block = case["batch"], case["hkv"], case["d"], case["block"]
    sel = s["sel"].long()
    cap = sel.shape[2]
    pages = s["table"].long().gather(2, sel.clamp(min=0)).clamp(min=0)
    at = sel[..., None] * block + torch.arange(block, device=DEV)
    there = ((at < s["seq_lens"].long()[:, None, None, None])
             & (torch.arange(cap, device=DEV)[:, None] < s["sel_count"][..., None, None])).view(batch, hkv, 1, -1)
    q = s["q"].float().view(batch, hkv, -1, d)
    k = (s["k"][pages].float() * s["k_scales"][pages][..., None, None]).view(batch, hkv, -1, d)
    logits = (q @ k.transpose(2, 3)) / math.sqrt(d)
    del k
    logits = logits.masked_fill(~there, -math.inf)
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - m)
    total = p.sum(-1, keepdim=True)
    v = (s["v"][pages].float() * s["v_scales"][pages][..., None, None]).view(batch, hkv, -1, d)
    out = ((p @ v) / total).to(torch.bfloat16).view(batch, -1, d)
    return {"out": out, "lse": (m + torch.log(total)).view(batch, -1)}


def _summaries_plain(s):
    lo, hi = _page_summaries(s, "fp8_block", s["seq_lens"].long())
    return {"smin": lo, "smax": hi}


# ---- the library's calls -------------------------------------------------------------------------------------------------


def _describe(s):
    from query_aware_sparse_hs_gb300 import hs
    case = s["case"]
    p = s["plan"] = {"shape": hs.attn_shape(case["hq"], case["hkv"], case["d"], case["block"], s["kind"])}
    p["kv"] = hs.paged_kv(s["k"], s["v"], s["table"], s["seq_lens"], s["k_scales"], s["v_scales"])
    if case["op"] == "append":
        p["params"] = hs.append_params(cos_sin=s["cos_sin"], interleaved=case["interleaved"], new_offsets=s["offsets"])
    elif case["op"] == "attend":
        p["counters"] = torch.zeros(case["batch"] * case["hkv"], dtype=torch.int32, device=DEV)
        p["params"] = hs.attn_params(1.0 / math.sqrt(case["d"]), split_counters=p["counters"])
        need = hs.hs_workspace_bytes(p["shape"], case["batch"], s["sel"].shape[2], p["params"])
        p["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)


def _call(s):
    from query_aware_sparse_hs_gb300 import hs
    p, op = s["plan"], s["case"]["op"]
    if op == "append":
        hs.hs_append_tokens(p["shape"], p["kv"], p["params"], s["k_new"], s["v_new"], s["q"], s["q_out"], s["smin"], s["smax"])
        return _append_out(s)
    if op == "attend":
        hs.hs_sparse_paged_decode_attn(p["shape"], p["kv"], s["q"], s["sel"], s["sel_count"], s["sel"].shape[2], p["params"],
                                       s["out"], s["lse"], p["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    hs.hs_build_block_summaries(p["shape"], p["kv"], 0, s["smin"], s["smax"])
    return {"smin": s["smin"], "smax": s["smax"]}


def run(state):
    if own:
        return _call(state)
    return {"append": _append_plain, "attend": _attend_plain, "summaries": _summaries_plain}[state["case"]["op"]](state)


# ---- from the definition, in 64 bits -------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"append": _append_exact, "attend": _attend_exact, "summaries": _summaries_exact}[case["op"]](s)


def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _to_bf16_below(x):
    """The largest bf16 number at or below x, in 64 bits (values of ordinary size)."""
    _, e = torch.frexp(x)
    step = _power(e - 8)
    return torch.floor(x / step) * step


def _to_e4m3(x):
    """Nearest e4m3 number, ties to even, in 64 bits."""
    _, e = torch.frexp(x)
    step = _power(torch.clamp(e - 4, min=-9))
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _append_exact(s):
    case, kind = s["case"], s["kind"]
    block, rotary, inter, d, hkv = case["block"], case["rotary"], case["interleaved"], case["d"], case["hkv"]
    if sum(_new(case)) * case["hq"] * d > 3e8 or _touched(case) > 4000:
        return None  # would take long
    h = rotary // 2
    i = torch.arange(h, device=DEV)
    first, second = (2 * i, 2 * i + 1) if inter else (i, i + h)

    def turned(x, p):
        c, sn = s["cos_sin"][p, :h].double(), s["cos_sin"][p, h:].double()
        y = x.double().clone()
        y[..., first] = x[..., first].double() * c[:, None] - x[..., second].double() * sn[:, None]
        y[..., second] = x[..., second].double() * c[:, None] + x[..., first].double() * sn[:, None]
        return y

    q = s["q_out"].double()
    held = {w: s[w].double() for w in ("k", "v")}
    scales = {w: None if s[w + "_scales"] is None else s[w + "_scales"].double() for w in ("k", "v")}
    smin, smax = (None, None) if s["smin"] is None else (s["smin"].double(), s["smax"].double())
    row = 0
    for b, (L, n) in enumerate(zip(_seq_lens(case), _new(case))):
        if n == 0:
            continue
        p = torch.arange(L - n, L, device=DEV)
        q[row:row + n] = turned(s["q"][row:row + n], p)
        fresh = {"k": turned(s["k_new"][row:row + n], p), "v": s["v_new"][row:row + n].double()}
        row += n
        for j in range((L - n) // block, -(-L // block)):
            a, z = max(L - n, j * block), min(L, (j + 1) * block)
            r0, r1 = a - j * block, z - j * block
            page = s["table"][b, :, j].long()
            for w in ("k", "v"):
                x = fresh[w][a - (L - n):z - (L - n)].transpose(0, 1)  # [hkv, rows, d]
                if kind == "fp8_block":
                    amax = x.abs().amax((1, 2))
                    near = torch.log2(amax / E4M3_MAX).round().clamp(min=MIN_SCALE_EXP)  # 2^near or its neighbour above
                    want = torch.where(amax > E4M3_MAX * _power(near), _power(near + 1), _power(near))
                    have = scales[w][page]
                    now = torch.maximum(have, want) if r0 else want
                    if r0:
                        held[w][page, :r0] = _to_e4m3(held[w][page, :r0] * (have / now)[:, None, None])
                    scales[w][page] = now
                    x = _to_e4m3(x / now[:, None, None])
                elif kind == "fp8":
                    grp = x.unflatten(-1, (-1, 32))
                    top = grp.abs().amax(-1)
                    sc = torch.where(top > 0, top / E4M3_MAX, 1.0).float().double()  # the scale is a 32-bit number
                    scales[w][page, r0:r1] = sc
                    x = _to_e4m3(grp / sc[..., None]).flatten(-2)
                held[w][page, r0:r1] = x
            if smin is not None:
                y = held["k"][page, :r1]
                if kind == "fp8_block":
                    y = y * scales["k"][page][:, None, None]
                elif kind == "fp8":
                    y = y * scales["k"][page, :r1].repeat_interleave(32, -1)
                elif kind == "bf16":
                    y = y.to(torch.bfloat16).double()
                lo, hi = y.amin(1), y.amax(1)
                smin[b, :, j], smax[b, :, j] = (lo, hi) if kind == "f32" else (_to_bf16_below(lo), -_to_bf16_below(-hi))
    return {"q_out": q, "k": held["k"], "v": held["v"], "k_scales": scales["k"], "v_scales": scales["v"], "smin": smin, "smax": smax}


def _attend_exact(s):
    case = s["case"]
    hkv, d, block = case["hkv"], case["d"], case["block"]
    if sum(_attended(case)) * hkv * d > 1.2e9:
        return None  # would take long
    grp = case["hq"] // hkv
    out = torch.zeros((case["batch"], case["hq"], d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((case["batch"], case["hq"]), dtype=torch.float64, device=DEV)
    counts, lens = s["sel_count"].tolist(), _seq_lens(case)
    for b in range(case["batch"]):
        for h in range(hkv):
            sel = s["sel"][b, h, :counts[b][h]].long()
            page = s["table"][b, h, sel].long()
            live = (sel[:, None] * block + torch.arange(block, device=DEV) < lens[b]).flatten()
            k = (s["k"][page].double() * s["k_scales"][page].double()[:, None, None]).view(-1, d)[live]
            v = (s["v"][page].double() * s["v_scales"][page].double()[:, None, None]).view(-1, d)[live]
            z = s["q"][b, h * grp:(h + 1) * grp].double() @ k.T * d ** -0.5
            lse[b, h * grp:(h + 1) * grp] = torch.logsumexp(z, -1)
            out[b, h * grp:(h + 1) * grp] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}


def _summaries_exact(s):
    case = s["case"]
    block = case["block"]
    smin, smax = s["smin"].double(), s["smax"].double()
    for b, L in enumerate(_seq_lens(case)):
        for h in range(case["hkv"]):
            whole, rest = divmod(L, block)
            page = s["table"][b, h, :-(-L // block)].long()
            x = s["k"][page].double() * s["k_scales"][page].double()[:, None, None]
            lo, hi = x.amin(1), x.amax(1)
            if rest:
                lo[whole], hi[whole] = x[whole, :rest].amin(0), x[whole, :rest].amax(0)
            smin[b, h, :len(page)], smax[b, h, :len(page)] = _to_bf16_below(lo), -_to_bf16_below(-hi)
    return {"smin": smin, "smax": smax}
