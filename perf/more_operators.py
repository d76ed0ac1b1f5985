"""A paged cache held in 4 bits (its append, attention and block summaries), attention weights accumulated per token, and the
eviction of the lightest tokens: the cases that are measured, their plain forms, and the library's calls for them.

A cache of kind ``int4`` holds, for every token and 32 channels, a bf16 scale s, a bf16 centre z and codes c of -8 .. 7 (stored
as c + 8, two to a byte): a value is z + s c.
"""

import math
import random

import torch

own = False

DEV = "cuda"
MOST = 2.0 ** 126  # values beyond it are held as it


def _append(name, batch, hq, hkv, d, block, ctx_min, ctx_max, new_min, new_max, rotary, interleaved, summaries):
    c = {"op": "append", "kind": "int4", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max, "new_min": new_min, "new_max": new_max, "rotary": rotary, "interleaved": interleaved,
         "summaries": summaries}
    return dict(c, name=name) if name else c


def _attend(name, batch, hq, hkv, d, block, ctx_min, ctx_max, keep):
    c = {"op": "attend", "kind": "int4", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max, "keep": keep}
    return dict(c, name=name) if name else c


def _summaries(name, batch, hq, hkv, d, block, ctx_min, ctx_max):
    c = {"op": "summaries", "kind": "int4", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max}
    return dict(c, name=name) if name else c


def _weights(name, kind, batch, hq, hkv, d, block, ctx_min, ctx_max, keep):
    c = {"op": "weights", "kind": kind, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max, "keep": keep}
    return dict(c, name=name) if name else c


def _evict(name, kind, batch, hq, hkv, d, block, ctx_min, ctx_max, budget, sink, recent):
    c = {"op": "evict", "kind": kind, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "block": block, "ctx_min": ctx_min,
         "ctx_max": ctx_max, "budget": budget, "sink": sink, "recent": recent}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token of each of a few short requests: latency counts
        _append("append_tokens_b8", 8, 32, 4, 128, 64, 30, 300, 1, 1, 128, False, True),
        # prompts of a batch into the cache, behind nothing or a short prefix
        _append("append_prompts_8x4k", 8, 32, 4, 128, 64, 0, 130, 1000, 4096, 128, False, True),
        # one short request over its whole cache: the smallest
        _attend("attend_b1_500", 1, 32, 4, 128, 64, 500, 500, 0),
        # a decode batch over the selected 64 blocks of 131072-token requests (budget of 4096 tokens)
        _attend("attend_selected_b32", 32, 32, 4, 128, 64, 20000, 131072, 64),
        # 16 query heads to a kv head, 64 channels, uneven requests
        _attend("attend_g16_d64", 12, 32, 2, 64, 32, 3001, 40000, 0),
        # the largest: long requests over their whole caches
        _attend("attend_b16_131072", 16, 32, 4, 128, 64, 131072, 131072, 0),
        # summaries of a few short requests, and of a batch of long uneven ones with 16-token pages
        _summaries("summaries_b2_2500", 2, 32, 4, 128, 64, 1200, 2500),
        _summaries("summaries_b32_64k", 32, 32, 4, 128, 16, 4096, 65536),
        # weights of a decode step over a few short bf16 requests, and over whole long 4-bit caches
        _weights("weights_b4_3000_bf16", "bf16", 4, 32, 4, 128, 16, 37, 3000, 0),
        _weights("weights_b32_16384_int4", "int4", 32, 32, 4, 128, 64, 16384, 16384, 0),
        # two requests cut to 1024 tokens; a batch of long ones cut to 4096
        _evict("evict_b2_3000_int4", "int4", 2, 32, 4, 128, 64, 1500, 3000, 1024, 4, 256),
        _evict("evict_b16_32768_bf16", "bf16", 16, 32, 4, 128, 64, 3000, 32768, 4096, 4, 512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "summaries", "weights", "weights", "evict", "evict"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8, 8, 16])
    while hq > 32:
        hq //= 2
    block = rng.choice([16, 32, 64, 128, 16, 64, 48])
    batch = _log(rng, 1, 64)
    if op == "append":
        rotary = rng.choice([d, d, d // 2, 16])
        ctx = _log(rng, 1, 2000)
        if rng.random() < 0.4:
            return _append(None, batch, hq, hkv, d, block, rng.randrange(ctx), ctx, 1, 1, rotary, rng.random() < 0.3,
                           rng.random() < 0.8)
        new = _log(rng, 2, max(2, 32000 // batch))
        return _append(None, batch, hq, hkv, d, block, 0, min(ctx, 1000), rng.randrange(new), new, rotary, rng.random() < 0.3,
                       rng.random() < 0.8)
    most = min(131072, 8000000 // (hkv * d // 64) // batch // 2)
    kind = rng.choice(["int4", "int4", "bf16", "fp8", "fp8_block", "f32"])
    if kind == "f32":
        most //= 4
    ctx = _log(rng, 1, most)
    low = rng.randrange(max(1, ctx // 10), ctx + 1)
    if op == "attend":
        return _attend(None, batch, hq, hkv, d, block, low, ctx, rng.choice([0, 0, 8, 33, 64]))
    if op == "summaries":
        return _summaries(None, batch, hq, hkv, d, block, low, ctx)
    if op == "weights":
        return _weights(None, kind, batch, hq, hkv, d, block, low, ctx, rng.choice([0, 0, 8, 33, 64]))
    budget = _log(rng, 1, max(2, ctx))
    sink = rng.choice([0, 1, 4]) if budget >= 8 else 0
    return _evict(None, rng.choice(["int4", "bf16", "fp8", "f32"]) if kind == "fp8_block" else kind, batch, hq, hkv, d, block,
                  low, ctx, budget, sink, rng.randrange(budget - sink + 1))


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


def _row_bytes(case):
    """A token's K (or V) of one kv head as the cache holds it."""
    return {"f32": 4.0, "bf16": 2.0, "fp8": 1.125, "fp8_block": 1.0, "int4": 0.625}[case["kind"]] * case["d"]


def work(case):
    hq, hkv, d, batch, op = case["hq"], case["hkv"], case["d"], case["batch"], case["op"]
    row = _row_bytes(case)
    if op == "append":
        rows, held = sum(_new(case)), sum(_seq_lens(case))
        # rows in and out, angles, boxes; and the whole cache read back as the values it stands for
        b = rows * ((2 * hq + 2 * hkv) * d * 2 + 2 * hkv * row + case["rotary"] * 4) + 8 * batch + 2 * held * hkv * (row + 2 * d)
        if case["summaries"]:
            b += _touched(case) * hkv * 2 * d * 2
        return {"bytes": b, "flops": rows * (hq + hkv) * case["rotary"] * 3}
    if op in ("attend", "weights"):
        tokens = sum(_attended(case))
        sel = sum(-(-n // case["block"]) for n in _attended(case))
        wide = 4 if case["kind"] == "f32" else 2
        if op == "weights":
            return {"bytes": tokens * hkv * (row + 8) + sel * hkv * 8 + batch * hq * (wide * d + 4), "flops": tokens * hq * d * 2}
        return {"bytes": tokens * hkv * 2 * row + sel * hkv * 8 + batch * hq * (4 * d + 4), "flops": tokens * hq * d * 4}
    if op == "summaries":
        return {"bytes": hkv * (sum(_seq_lens(case)) * row + sum(_blocks(case)) * (4 * d + 4)), "flops": sum(_seq_lens(case)) * hkv * d * 4}
    kept = sum(min(L, case["budget"]) for L in _seq_lens(case))
    b = hkv * (sum(L for L in _seq_lens(case) if L > case["budget"]) * 4 + kept * (4 * row + 12)) + 8 * batch
    if case["kind"] == "int4":  # the new pages read back
        b += 2 * kept * hkv * (row + 2 * d)
    return {"bytes": b, "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------------------------------


def _pool(case, blocks, g):
    """Page table of so many blocks of every request over a shuffled pool with spare pages."""
    hkv = case["hkv"]
    mb = max(1, max(blocks))
    used = sum(blocks) * hkv
    pages = used + 3
    order = torch.randperm(pages, generator=g, device=DEV)[:used].to(torch.int32)
    nb = torch.tensor(blocks, device=DEV)
    there = (torch.arange(mb, device=DEV)[None, None, :] < nb[:, None, None]).expand(case["batch"], hkv, mb)
    table = torch.full((case["batch"], hkv, mb), -1, dtype=torch.int32, device=DEV)
    table[there] = order
    return table, pages


def _cache(case, g):
    """Pages with values in them, and the scales that go with the codes."""
    kind = case["kind"]
    table, pages = _pool(case, _blocks(case), g)
    shape = (pages, case["block"], case["d"])
    s = {"table": table, "k_scales": None, "v_scales": None}
    for w in ("k", "v"):
        if kind == "f32":
            s[w] = torch.randn(shape, generator=g, device=DEV)
        elif kind == "bf16":
            s[w] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        elif kind == "fp8":
            s[w] = (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[w + "_scales"] = 0.004 + 0.012 * torch.rand(shape[:2] + (case["d"] // 32,), generator=g, device=DEV)
        elif kind == "fp8_block":
            s[w] = (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[w + "_scales"] = torch.exp2(torch.randint(-8, -5, (pages,), generator=g, device=DEV).float())
        else:  # ranges of about four deviations around centres near zero
            s[w] = torch.randint(0, 256, shape[:2] + (case["d"] // 2,), generator=g, device=DEV, dtype=torch.uint8)
            sc = 0.2 + 0.15 * torch.rand(shape[:2] + (1, case["d"] // 32), generator=g, device=DEV)
            z = 0.3 * torch.randn(shape[:2] + (1, case["d"] // 32), generator=g, device=DEV)
            s[w + "_scales"] = torch.cat([sc, z], 2).to(torch.bfloat16)
    return s


def _values(codes, scales):
    """What 4-bit rows stand for, in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    s, z = scales.float().unbind(-2)
    return (c.float() - 8.0).unflatten(-1, (-1, 32)).mul_(s[..., None]).add_(z[..., None]).flatten(-2)


def _held(s, w, pages=slice(None)):
    """What the pages stand for, in 32 bits."""
    kind, x, scales = s["kind"], s[w][pages], s[w + "_scales"]
    if kind == "int4":
        return _values(x, scales[pages])
    if kind == "fp8":
        return x.float() * scales[pages].repeat_interleave(32, -1)
    return x.float() * scales[pages][..., None, None] if kind == "fp8_block" else x.float()


def _outward(lo, hi):
    """bf16 bounds at or below lo, at or above hi (finite values)."""
    def down(x):
        y = x.to(torch.bfloat16)
        return torch.where(y.double() > x.double(), torch.nextafter(y, torch.full_like(y, -math.inf)), y)
    return down(lo), -down(-hi)


def _wide(kind):
    return torch.float32 if kind == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    batch, hq, hkv, d, block, kind, op = (case[k] for k in ("batch", "hq", "hkv", "d", "block", "kind", "op"))
    s = {"case": dict(case), "kind": kind}
    s.update(_cache(case, g))
    seq = _seq_lens(case)
    s["seq_lens"] = torch.tensor(seq, dtype=torch.int32, device=DEV)
    mb = s["table"].shape[2]
    if op == "append":
        new = _new(case)
        rows = sum(new) + _pad_rows(case)
        # the rows of a fused projection: q, k and v are views of it
        qkv = (torch.randn((rows, hq + 2 * hkv, d), generator=g, device=DEV) * 1.3).to(torch.bfloat16)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=DEV)
        one = case["new_min"] == case["new_max"] == 1
        s["offsets"] = None if one else torch.tensor([sum(new[:i]) for i in range(batch + 1)], dtype=torch.int32, device=DEV)
        h = case["rotary"] // 2
        inv = 10000.0 ** (-torch.arange(h, device=DEV, dtype=torch.float64) / h)
        angle = torch.arange(max(1, max(seq)), device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["smin"] = s["smax"] = None
        if case["summaries"]:  # of what the cache holds before the new tokens
            lo, hi = _page_summaries(s, torch.tensor([L - n for L, n in zip(seq, new)], device=DEV))
            s["smin"], s["smax"] = lo.contiguous(), hi.contiguous()
        s["values"] = {w: torch.zeros(s[w].shape[:2] + (d,), dtype=torch.bfloat16, device=DEV) for w in ("k", "v")}
    elif op in ("attend", "weights"):
        s["q"] = torch.randn((batch, hq, d), generator=g, device=DEV).to(_wide(kind))
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
        if op == "attend":
            s["out"] = torch.empty((batch, hq, d), dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty((batch, hq), dtype=torch.float32, device=DEV)
        else:  # what the step's attention left, and the weights of the steps before
            s["lse"] = torch.logsumexp(_logits(s)[0], -1).view(batch, hq).contiguous()
            s["weights"] = torch.rand((batch, hkv, mb * block), generator=g, device=DEV) ** 4
    elif op == "summaries":
        s["smin"] = torch.zeros((batch, hkv, mb, d), dtype=torch.bfloat16, device=DEV)
        s["smax"] = torch.zeros_like(s["smin"])
    else:
        x = torch.rand((batch, hkv, mb * block), generator=g, device=DEV)
        s["weights"] = torch.where(x < 0.1, torch.zeros_like(x), x ** 6)  # a few tokens never looked at
        left = [-(-min(L, case["budget"]) // block) for L in seq]
        s["dst_table"], pages = _pool(case, left, g)
        for w in ("k", "v"):
            s["dst_" + w] = torch.zeros((pages,) + s[w].shape[1:], dtype=s[w].dtype, device=DEV)
            sc = s[w + "_scales"]
            s["dst_" + w + "_scales"] = None if sc is None else torch.zeros((pages,) + sc.shape[1:], dtype=sc.dtype, device=DEV)
            if kind == "int4":
                s["dst_" + w + "_values"] = torch.zeros((pages, block, d), dtype=torch.bfloat16, device=DEV)
        s["dst_weights"] = torch.zeros((batch, hkv, s["dst_table"].shape[2] * block), device=DEV)
        s["dst_lens"] = torch.zeros(batch, dtype=torch.int32, device=DEV)
        s["kept"] = torch.zeros((batch, hkv, case["budget"]), dtype=torch.int32, device=DEV)
    if own:  # the descriptors and the workspace that a program keeps from step to step
        _describe(s)
    return s


# ---- plain forms ---------------------------------------------------------------------------------------------------------


def _page_summaries(s, lens):
    """min / max over the first `lens` tokens of every request, by block; 0 where a block has none."""
    table = s["table"].long()
    batch, hkv, mb = table.shape
    block = s["k"].shape[1]
    valid = (lens[:, None, None] - torch.arange(mb, device=DEV) * block).clamp(0, block).expand(batch, hkv, mb)
    there = valid > 0
    count = torch.zeros(s["k"].shape[0], dtype=torch.long, device=DEV)
    count[table[there]] = valid[there]
    gone = torch.arange(block, device=DEV)[None, :, None] >= count[:, None, None]
    x = _held(s, "k")
    lo, hi = _outward(x.masked_fill(gone, math.inf).amin(1), x.masked_fill_(gone, -math.inf).amax(1))
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


def _quantise(x):
    """Codes (two to a byte) and scales of rows, in 64 bits: values next to a border."""
    x = x.clamp(-MOST, MOST).unflatten(-1, (-1, 32))
    lo, hi = x.amin(-1), x.amax(-1)
    z = ((7 * lo + 8 * hi) / 15).to(torch.bfloat16)
    zd = z.double()
    top = torch.maximum((hi - zd) / 7, (zd - lo) / 8)
    sc = -_outward(-top, -top)[0]
    sd = sc.double()[..., None]
    c = torch.where(sd > 0, torch.round((x - zd[..., None]) / torch.where(sd > 0, sd, 1.0)), 0.0)
    c = (c.clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([sc, z], -2)


def _append_plain(s):
    case = s["case"]
    rotary, inter, block = case["rotary"], case["interleaved"], case["block"]
    req, pos, real = _rows(s)
    cos, sin = s["cos_sin"][pos.clamp(0, len(s["cos_sin"]) - 1)].split(rotary // 2, 1)
    q = _rotate(s["q"].float(), cos, sin, rotary, inter).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(real[:, None, None], q, s["q_out"]))
    req, pos = req[real], pos[real]
    j, r = pos // block, pos % block
    pages = s["table"].long()[req, :, j]  # [rows, hkv]
    k = _rotate(s["k_new"].double(), cos.double(), sin.double(), rotary, inter)[real]
    for w, x in (("k", k), ("v", s["v_new"].double()[real])):
        codes, scales = _quantise(x)
        s[w][pages, r[:, None]] = codes
        s[w + "_scales"][pages, r[:, None]] = scales
    if s["smin"] is not None:
        lo, hi = _page_summaries(s, s["seq_lens"].long())
        mb = s["table"].shape[2]
        n = torch.bincount(req, minlength=s["table"].shape[0])
        start = (s["seq_lens"].long() - n) // block
        cols = torch.arange(mb, device=DEV)[None]
        mine = ((n > 0)[:, None] & (cols >= start[:, None]) & (cols * block < s["seq_lens"][:, None]))[:, None, :, None]
        s["smin"].copy_(torch.where(mine, lo, s["smin"]))
        s["smax"].copy_(torch.where(mine, hi, s["smax"]))
    for w in ("k", "v"):
        s["values"][w].copy_(_held(s, w))
    return _append_out(s)


def _append_out(s):
    return {"q_out": s["q_out"], "k": s["values"]["k"], "v": s["values"]["v"], "smin": s["smin"], "smax": s["smax"]}


def _logits(s):
    """Logits [batch][hkv][group][tokens] of the selected blocks (-inf where there is none), pages and positions."""
    case = s["case"]
    batch, hkv, d, block = case["batch"], case["hkv"], case["d"], case["block"]
    sel = s["sel"].long()
    pages = s["table"].long().gather(2, sel.clamp(min=0)).clamp(min=0)
    at = sel[..., None] * block + torch.arange(block, device=DEV)
    there = ((at < s["seq_lens"].long()[:, None, None, None])
             & (torch.arange(sel.shape[2], device=DEV)[:, None] < s["sel_count"][..., None, None])).view(batch, hkv, -1)
    q = s["q"].float().view(batch, hkv, -1, d)
    k = _held(s, "k", pages).view(batch, hkv, -1, d)
    logits = (q @ k.transpose(2, 3)) / math.sqrt(d)
    return logits.masked_fill(~there[:, :, None], -math.inf), pages, at.view(batch, hkv, -1), there


def _attend_plain(s):
    case = s["case"]
    logits, pages, _, _ = _logits(s)
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - m)
    total = p.sum(-1, keepdim=True)
    v = _held(s, "v", pages).view(case["batch"], case["hkv"], -1, case["d"])
    out = ((p @ v) / total).to(torch.bfloat16).view(case["batch"], -1, case["d"])
    return {"out": out, "lse": (m + torch.log(total)).view(case["batch"], -1)}


def _summaries_plain(s):
    lo, hi = _page_summaries(s, s["seq_lens"].long())
    return {"smin": lo, "smax": hi}


def _weights_plain(s):
    case = s["case"]
    logits, _, at, there = _logits(s)
    lse = s["lse"].view(case["batch"], case["hkv"], -1, 1)
    add = torch.exp(logits - lse).sum(2)
    s["weights"].scatter_add_(2, torch.where(there, at, 0), torch.where(there, add, 0.0))
    return {"weights": s["weights"]}


def _evict_plain(s):
    case = s["case"]
    block, budget, hkv, batch = case["block"], case["budget"], case["hkv"], case["batch"]
    L = s["seq_lens"].long()[:, None, None]
    n = s["weights"].shape[2]
    t = torch.arange(n, device=DEV)
    forced = (t < case["sink"]) | (t >= L - case["recent"])
    # forced tokens first, then the others by weight (the sort is stable: lower indices first), then what is not there
    rank = torch.where(forced, math.inf, s["weights"]).masked_fill(t >= L, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order, (0, budget - order.shape[2]), value=n)
    left = L.clamp(max=budget)
    i = torch.arange(budget, device=DEV)
    at = torch.where(i < left, order, n).sort(-1).values
    s["kept"].copy_(torch.where(i < left, at, -1))
    s["dst_lens"].copy_(left.view(-1))
    there = (i < left).expand(batch, hkv, budget)
    b, h, i = there.nonzero(as_tuple=True)
    src = at[b, h, i]
    from_page, to_page = s["table"].long()[b, h, src // block], s["dst_table"].long()[b, h, i // block]
    s["dst_weights"][b, h, i] = s["weights"][b, h, src]
    for w in ("k", "v", "k_scales", "v_scales"):
        if s[w] is not None:
            x, y = s[w], s["dst_" + w]
            if x.dtype == torch.float8_e4m3fn:
                x, y = x.view(torch.uint8), y.view(torch.uint8)
            y[to_page, i % block] = x[from_page, src % block]
    if s["kind"] == "int4":
        for w in ("k", "v"):
            s["dst_" + w + "_values"].copy_(_values(s["dst_" + w], s["dst_" + w + "_scales"]))
    return _evict_out(s)


def _evict_out(s):
    out = {"kept": s["kept"], "lens": s["dst_lens"], "weights": s["dst_weights"]}
    for w in ("k", "v"):
        out[w] = s["dst_" + w + "_values"] if s["kind"] == "int4" else s["dst_" + w]
        out[w + "_scales"] = None if s["kind"] == "int4" else s["dst_" + w + "_scales"]
    return out


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
    elif case["op"] == "evict":
        p["dst"] = hs.paged_kv(s["dst_k"], s["dst_v"], s["dst_table"], s["dst_lens"], s["dst_k_scales"], s["dst_v_scales"])
        p["params"] = hs.evict_params(case["budget"], case["sink"], case["recent"])


def _call(s):
    from query_aware_sparse_hs_gb300 import hs
    p, op = s["plan"], s["case"]["op"]
    if op == "append":
        hs.hs_append_tokens(p["shape"], p["kv"], p["params"], s["k_new"], s["v_new"], s["q"], s["q_out"], s["smin"], s["smax"])
        for w in ("k", "v"):
            hs.hs_dequantize_int4_g32(s[w], s[w + "_scales"], s["values"][w])
        return _append_out(s)
    if op == "attend":
        hs.hs_sparse_paged_decode_attn(p["shape"], p["kv"], s["q"], s["sel"], s["sel_count"], s["sel"].shape[2], p["params"],
                                       s["out"], s["lse"], p["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "summaries":
        hs.hs_build_block_summaries(p["shape"], p["kv"], 0, s["smin"], s["smax"])
        return {"smin": s["smin"], "smax": s["smax"]}
    if op == "weights":
        hs.hs_accumulate_attn_weights(p["shape"], p["kv"], s["q"], s["lse"], s["sel"], s["sel_count"], s["sel"].shape[2],
                                      1.0 / math.sqrt(s["case"]["d"]), s["weights"])
        return {"weights": s["weights"]}
    hs.hs_evict_tokens(p["shape"], p["kv"], p["dst"], p["params"], s["weights"], s["dst_weights"], s["kept"])
    if s["kind"] == "int4":
        for w in ("k", "v"):
            hs.hs_dequantize_int4_g32(s["dst_" + w], s["dst_" + w + "_scales"], s["dst_" + w + "_values"])
    return _evict_out(s)


def run(state):
    if own:
        return _call(state)
    op = state["case"]["op"]
    return {"append": _append_plain, "attend": _attend_plain, "summaries": _summaries_plain, "weights": _weights_plain,
            "evict": _evict_plain}[op](state)


# ---- from the definition, in 64 bits -------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"append": _append_exact, "attend": _attend_exact, "summaries": _summaries_exact, "weights": _weights_exact,
                "evict": _evict_exact}[case["op"]](s)


def _row64(s, w, page):
    """Values [.., block, d] of pages, in 64 bits."""
    x = s[w][page]
    if s["kind"] == "int4":
        y = torch.empty(x.shape[:-1] + (2 * x.shape[-1],), dtype=torch.float64, device=DEV)
        y[..., 0::2], y[..., 1::2] = (x % 16).double() - 8, (x // 16).double() - 8
        sc = s[w + "_scales"][page].double()
        return y * sc[..., 0, :].repeat_interleave(32, -1) + sc[..., 1, :].repeat_interleave(32, -1)
    x = x.double()
    if s["kind"] == "fp8":
        return x * s[w + "_scales"][page].double().repeat_interleave(32, -1)
    return x * s[w + "_scales"][page].double()[..., None, None] if s["kind"] == "fp8_block" else x


def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _to_bf16(x, how):
    """x rounded to 8 significant bits by `how`, in 64 bits (values of ordinary size)."""
    _, e = torch.frexp(x)
    step = _power(e - 8)
    return how(x / step) * step


def _append_exact(s):
    case = s["case"]
    block, rotary, inter = case["block"], case["rotary"], case["interleaved"]
    if sum(_new(case)) * case["hq"] * case["d"] > 3e8 or _touched(case) > 4000:
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

    def held_as(x):
        grp = x.unflatten(-1, (-1, 32))
        lo, hi = grp.amin(-1, keepdim=True), grp.amax(-1, keepdim=True)
        z = _to_bf16(lo + (hi - lo) * 8 / 15, torch.round)
        sc = _to_bf16(torch.maximum((hi - z) / 7, (z - lo) / 8), torch.ceil)
        return (z + sc * ((grp - z) / sc).round().clamp(-8, 7)).flatten(-2)

    q = s["q_out"].double()
    every = slice(None)
    held = {w: _row64(s, w, every) for w in ("k", "v")}
    smin, smax = (None, None) if s["smin"] is None else (s["smin"].double(), s["smax"].double())
    row = 0
    for b, (L, n) in enumerate(zip(_seq_lens(case), _new(case))):
        if n == 0:
            continue
        p = torch.arange(L - n, L, device=DEV)
        q[row:row + n] = turned(s["q"][row:row + n], p)
        fresh = {"k": held_as(turned(s["k_new"][row:row + n], p)), "v": held_as(s["v_new"][row:row + n].double())}
        row += n
        for j in range((L - n) // block, -(-L // block)):
            a, z = max(L - n, j * block), min(L, (j + 1) * block)
            r0, r1 = a - j * block, z - j * block
            page = s["table"][b, :, j].long()
            for w in ("k", "v"):
                held[w][page, r0:r1] = fresh[w][a - (L - n):z - (L - n)].transpose(0, 1)
            if smin is not None:
                y = held["k"][page, :r1].float().double()  # the boxes are of 32-bit values
                smin[b, :, j], smax[b, :, j] = _to_bf16(y.amin(1), torch.floor), _to_bf16(y.amax(1), torch.ceil)
    return {"q_out": q, "k": held["k"], "v": held["v"], "smin": smin, "smax": smax}


def _each_pair(s):
    """(request, kv head, 64-bit values of the selected K rows, their pages' rows, positions) of every pair."""
    case = s["case"]
    block, counts, lens = case["block"], s["sel_count"].tolist(), _seq_lens(case)
    for b in range(case["batch"]):
        for h in range(case["hkv"]):
            sel = s["sel"][b, h, :counts[b][h]].long()
            page = s["table"][b, h, sel].long()
            at = (sel[:, None] * block + torch.arange(block, device=DEV)).flatten()
            yield b, h, page, at, at < lens[b]


def _attend_exact(s):
    case = s["case"]
    d = case["d"]
    if sum(_attended(case)) * case["hkv"] * d > 1.2e9:
        return None  # would take long
    grp = case["hq"] // case["hkv"]
    out = torch.zeros((case["batch"], case["hq"], d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((case["batch"], case["hq"]), dtype=torch.float64, device=DEV)
    for b, h, page, _, live in _each_pair(s):
        k, v = (_row64(s, w, page).view(-1, d)[live] for w in ("k", "v"))
        z = s["q"][b, h * grp:(h + 1) * grp].double() @ k.T * d ** -0.5
        lse[b, h * grp:(h + 1) * grp] = torch.logsumexp(z, -1)
        out[b, h * grp:(h + 1) * grp] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}


def _weights_exact(s):
    case = s["case"]
    d = case["d"]
    if sum(_attended(case)) * case["hkv"] * d > 1.2e9:
        return None  # would take long
    grp = case["hq"] // case["hkv"]
    w = s["weights"].double()
    for b, h, page, at, live in _each_pair(s):
        z = _row64(s, "k", page).view(-1, d)[live] @ s["q"][b, h * grp:(h + 1) * grp].double().T * d ** -0.5
        w[b, h, at[live]] += torch.exp(z - s["lse"][b, h * grp:(h + 1) * grp].double()).sum(1)
    return {"weights": w}


def _summaries_exact(s):
    case = s["case"]
    block = case["block"]
    smin, smax = s["smin"].double(), s["smax"].double()
    for b, L in enumerate(_seq_lens(case)):
        for h in range(case["hkv"]):
            whole, rest = divmod(L, block)
            page = s["table"][b, h, :-(-L // block)].long()
            x = _row64(s, "k", page).float().double()  # the boxes are of 32-bit values
            lo, hi = x.amin(1), x.amax(1)
            if rest:
                lo[whole], hi[whole] = x[whole, :rest].amin(0), x[whole, :rest].amax(0)
            smin[b, h, :len(page)], smax[b, h, :len(page)] = _to_bf16(lo, torch.floor), _to_bf16(hi, torch.ceil)
    return {"smin": smin, "smax": smax}


def _evict_exact(s):
    case = s["case"]
    block, budget = case["block"], case["budget"]
    if case["batch"] * case["hkv"] > 600:
        return None  # would take long
    out = {"kept": None, "lens": None, "weights": s["dst_weights"].double()}
    for w in ("k", "v"):
        pages = s["dst_" + w].shape[0]
        out[w] = torch.zeros((pages, block, case["d"]), dtype=torch.float64, device=DEV)
        out[w + "_scales"] = s["dst_" + w + "_scales"].double() if s["kind"] == "fp8" else None
    for b, L in enumerate(_seq_lens(case)):
        for h in range(case["hkv"]):
            t = torch.arange(L, device=DEV)
            if L > budget:
                free = t[case["sink"]:L - case["recent"]]
                x = s["weights"][b, h, free]
                need = budget - case["sink"] - case["recent"]
                cut = x.sort(descending=True).values[need - 1] if need else math.inf
                above = x > cut
                same = (x == cut).nonzero()[:, 0][:need - int(above.sum())]
                above[same] = True
                t = torch.cat([t[:case["sink"]], free[above], t[L - case["recent"]:]])
            i = torch.arange(len(t), device=DEV)
            src, dst = s["table"][b, h, t // block].long(), s["dst_table"][b, h, i // block].long()
            out["weights"][b, h, i] = s["weights"][b, h, t].double()
            for w in ("k", "v"):
                if s["kind"] == "int4":
                    x = {"kind": "int4", w: s[w][src, t % block], w + "_scales": s[w + "_scales"][src, t % block]}
                    out[w][dst, i % block] = _row64(x, w, slice(None))
                else:
                    out[w][dst, i % block] = s[w][src, t % block].double()
                    if s["kind"] == "fp8":
                        out[w + "_scales"][dst, i % block] = s[w + "_scales"][src, t % block].double()
    return out
