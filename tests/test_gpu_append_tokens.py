"""hs_append_tokens: rows of any number per request into f32, bf16, grouped and block-scaled e4m3 caches, rotated on the
way, against plain 64-bit loops; the summaries against the library's own builder and the plain min/max of what the cache
then holds.  GPU only."""

import math

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24  # half a step of fp32, relative
SENTINEL = 7.0


def power_scale(amax):
    """The smallest power of two s >= 2^-117 with amax <= 448 s."""
    if amax <= 448 * 2.0 ** -117:
        return 2.0 ** -117
    e = math.frexp(amax / 448)[1] - 1
    return 2.0 ** e if amax <= 448 * 2.0 ** e else 2.0 ** (e + 1)


def to_np(t):
    return t.detach().cpu().numpy() if t.dtype == torch.uint8 else t.detach().double().cpu().numpy()


class World:
    """A cache with earlier tokens in it and the rows of a fused projection."""

    def __init__(self, kind, d, block, hq, hkv, old, new, rotary, interleaved=False, positions=False, pad=0, seed=0,
                 spread=1.0, table=True):
        from query_aware_sparse_hs_gb300 import hs
        self.hs, self.kind, self.d, self.block, self.hq, self.hkv = hs, kind, d, block, hq, hkv
        self.old, self.new, self.rotary, self.interleaved = old, new, rotary, interleaved
        rng = np.random.default_rng(seed)
        self.batch = len(new)
        self.lens = [a + n for a, n in zip(old, new)]
        self.mb = max(1, max(-(-L // block) for L in self.lens)) + 1
        nb = [-(-L // block) for L in self.lens]
        self.pages = sum(nb) * hkv + 3
        order = rng.permutation(self.pages)
        self.table = np.full((self.batch, hkv, self.mb), -1, np.int32)
        at = 0
        for b in range(self.batch):
            for h in range(hkv):
                self.table[b, h, :nb[b]] = order[at:at + nb[b]]
                at += nb[b]
        shape = (self.pages, block, d)
        wide = torch.float32 if kind == "f32" else torch.bfloat16
        self.wide = wide
        f = lambda *s: torch.from_numpy(rng.standard_normal(s)).float()  # noqa: E731
        if kind.startswith("fp8"):
            self.cache = {w: torch.from_numpy(O.e4m3_encode(rng.standard_normal(shape) * 90)) for w in "kv"}
            s = (self.pages,) if kind == "fp8_block" else shape[:2] + (d // 32,)
            self.scales = {w: torch.from_numpy(np.exp2(rng.integers(-9, -5, s)).astype(np.float32)) for w in "kv"}
        else:
            self.cache = {w: f(*shape).to(wide) for w in "kv"}
            self.scales = {"k": None, "v": None}
        self.rows = sum(new) + pad
        qkv = (f(self.rows, hq + 2 * hkv, d) * torch.exp2(spread * f(self.rows, 1, 1))).to(wide)
        self.offsets = None if (pad == 0 and all(n == 1 for n in new)) else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.pos = rng.integers(0, 500, self.rows).astype(np.int32) if positions else None
        n_pos = max([500] + self.lens) if rotary else 1
        half = max(1, rotary // 2)
        ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(half) / half)
        self.cos_sin = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float()[:, :rotary].contiguous() if rotary else None
        dev = "cuda"
        self.g = {w: self.cache[w].to(dev).clone() for w in "kv"}
        self.gs = {w: None if self.scales[w] is None else self.scales[w].to(dev).clone() for w in "kv"}
        self.gt, self.gl = torch.from_numpy(self.table).to(dev), torch.tensor(self.lens, dtype=torch.int32, device=dev)
        g = qkv.to(dev)
        self.qkv = qkv.double().numpy()
        self.q, self.kn, self.vn = g[:, :hq], g[:, hq:hq + hkv], g[:, hq + hkv:]
        self.q_out = torch.full((self.rows, hq, d), SENTINEL, dtype=wide, device=dev)
        sdt = torch.float32 if kind == "f32" else torch.bfloat16
        self.smin = torch.full((self.batch, hkv, self.mb, d), SENTINEL, dtype=sdt, device=dev)
        self.smax = self.smin.clone()
        self.shape = hs.attn_shape(hq, hkv, d, block, kind)
        self.kv = hs.paged_kv(self.g["k"], self.g["v"], self.gt, self.gl, self.gs["k"], self.gs["v"])
        # summaries of the earlier tokens
        before = hs.paged_kv(self.g["k"], self.g["v"], self.gt, torch.tensor(old, dtype=torch.int32, device=dev),
                             self.gs["k"], self.gs["v"])
        hs.hs_build_block_summaries(self.shape, before, 0, self.smin, self.smax)
        self.params = hs.append_params(None if not rotary else self.cos_sin.to(dev), interleaved,
                                       None if self.offsets is None else torch.from_numpy(self.offsets).to(dev),
                                       None if self.pos is None else torch.from_numpy(self.pos).to(dev))

    def append(self, q=True, summaries=True, stream=None):
        self.hs.hs_append_tokens(self.shape, self.kv, self.params, self.kn, self.vn, self.q if q else None,
                                 self.q_out if q else None, self.smin if summaries else None,
                                 self.smax if summaries else None, stream)

    # ---- the definition, in 64 bits ----
    def turned(self, x, p):
        """x [heads][d] at position p, and per value the sum of magnitudes that bounds its fp32 error."""
        y, mag = x.copy(), np.abs(x)
        h = self.rotary // 2
        if h:
            c, s = self.cos_sin[p, :h].double().numpy(), self.cos_sin[p, h:].double().numpy()
            i = np.arange(h)
            a, b = (2 * i, 2 * i + 1) if self.interleaved else (i, i + h)
            y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
            mag = mag.copy()
            mag[:, a] = mag[:, b] = np.abs(x[:, a]) + np.abs(x[:, b])
        return y, mag

    def each_row(self):
        row = 0
        for b, (o, n) in enumerate(zip(self.old, self.new)):
            for i in range(n):
                t = o + i
                yield row, b, t, (int(self.pos[row]) if self.pos is not None else t)
                row += 1


# a product of fp32 numbers, a second one and their sum: three roundings of at most U32 of the magnitudes' sum
ARITH = 3 * U32


def check(w):
    """Everything hs_append_tokens leaves, against the definition."""
    hs = w.hs
    st, bits = hs.hs_get_device_error()
    assert st == hs.HS_OK, bits
    qo, held = to_np(w.q_out), {x: to_np(w.g[x]) for x in "kv"}
    scales = {x: None if w.gs[x] is None else to_np(w.gs[x]) for x in "kv"}
    half = U32 if w.kind == "f32" else 2.0 ** -8  # of the stored or returned type
    touched = {}  # page -> rows that were there before
    groups = {}   # page -> its new rows
    seen = np.zeros(w.rows, bool)
    for row, b, t, p in w.each_row():
        seen[row] = True
        y, mag = w.turned(w.qkv[row, :w.hq], p)
        assert (np.abs(qo[row] - y) <= half * np.abs(y) + (1 + half) * ARITH * mag).all(), (row, b, t)
        k, kmag = w.turned(w.qkv[row, w.hq:w.hq + w.hkv], p)
        v = w.qkv[row, w.hq + w.hkv:]
        j, r = divmod(t, w.block)
        for h in range(w.hkv):
            page = int(w.table[b, h, j])
            touched[page] = min(touched.get(page, w.block), r)
            groups.setdefault(page, []).append((r, k[h], kmag[h], v[h]))
    assert (qo[~seen] == SENTINEL).all()  # rows behind the last request
    for page in range(w.pages):
        if page not in touched:
            for x in "kv":
                assert torch.equal(w.g[x][page].cpu(), w.cache[x][page]), (page, x)
                if scales[x] is not None:
                    assert torch.equal(w.gs[x][page].cpu(), w.scales[x][page])
            continue
        first = touched[page]
        for x in "kv":
            codes0 = w.cache[x][page].numpy() if w.kind.startswith("fp8") else None
            rows = [(r, k, mag) if x == "k" else (r, v, np.zeros_like(v)) for r, k, mag, v in groups[page]]
            got = held[x][page]
            if w.kind in ("f32", "bf16"):
                for r, y, mag in rows:
                    assert (np.abs(got[r] - y) <= (half * np.abs(y) + (1 + half) * ARITH * mag if x == "k" else 0)).all(), (page, r, x)
                assert np.array_equal(got[:first], w.cache[x][page][:first].double().numpy())
                continue
            if w.kind == "fp8":
                for r, y, mag in rows:
                    s = scales[x][page, r]
                    top = np.abs(y).reshape(-1, 32).max(1)
                    want = np.where(top > 0, top / 448, 1.0)
                    # the amax carries ARITH of its magnitudes, the division one rounding
                    assert (np.abs(s - want) <= U32 * want + ARITH * mag.reshape(-1, 32).max(1) / 448 * (1 + U32)).all()
                    val = O.e4m3_decode(got[r]).reshape(-1, 32) * s[:, None]
                    yy = y.reshape(-1, 32)
                    # half a step of the code (2^-4 of the value, 2^-10 under the smallest normal), and the roundings before it
                    bound = np.maximum(2.0 ** -4 * np.abs(yy), 2.0 ** -10 * s[:, None]) * (1 + 4 * U32) + ARITH * mag.reshape(-1, 32) + 4 * U32 * np.abs(yy)
                    assert (np.abs(val - yy) <= bound).all(), (page, r, x)
                assert np.array_equal(got[:first], codes0[:first])
                continue
            # one power-of-two scale
            s = float(scales[x][page])
            top = max(np.abs(y).max() for _, y, _ in rows)
            slack = max((ARITH * mag).max() for _, _, mag in rows)
            allowed = {power_scale(max(top - slack, 0)), power_scale(top), power_scale(top + slack)}
            had = float(w.scales[x][page])
            if first:
                allowed = {max(had, z) for z in allowed}
            assert s in allowed, (page, x, s, allowed)
            if first:
                want = codes0[:first] if s == had else O.e4m3_encode((O.e4m3_decode(codes0[:first]) * (had / s)).astype(np.float32))
                assert np.array_equal(got[:first], want), (page, x)
            for r, y, mag in rows:
                if x == "v":
                    assert np.array_equal(got[r], O.e4m3_encode((y / s).astype(np.float32))), (page, r)
                val = O.e4m3_decode(got[r]) * s
                assert (np.abs(val - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) + (1 + 2.0 ** -4) * ARITH * mag).all(), (page, r, x)
    # rows of touched pages behind the last token stay as they were
    for b, L in enumerate(w.lens):
        if L % w.block and w.new[b]:
            for h in range(w.hkv):
                page = int(w.table[b, h, L // w.block])
                for x in "kv":
                    assert torch.equal(w.g[x][page, L % w.block:].cpu(), w.cache[x][page, L % w.block:])


def check_summaries(w):
    """Bit for bit what the builder computes over the cache as it is now, in the blocks of the new tokens and the others."""
    lo, hi = torch.full_like(w.smin, SENTINEL), torch.full_like(w.smax, SENTINEL)
    w.hs.hs_build_block_summaries(w.shape, w.kv, 0, lo, hi)
    assert torch.equal(w.smin, lo) and torch.equal(w.smax, hi)


CASES = {
    # kind, d, block, hq, hkv, earlier tokens, new tokens, rotary, interleaved, explicit positions, padding rows
    "tokens_block": ("fp8_block", 128, 64, 32, 4, [0, 63, 64, 130, 1], [1, 1, 1, 1, 1], 128, False, False, 0),
    "tokens_bf16": ("bf16", 128, 16, 8, 8, [15, 16, 300], [1, 1, 1], 128, False, False, 0),
    "tokens_g32": ("fp8", 64, 16, 16, 1, [0, 31], [1, 1], 64, True, False, 0),
    "tokens_padded": ("fp8_block", 64, 16, 4, 2, [3, 40], [1, 1], 32, False, False, 3),
    "prompts_block": ("fp8_block", 128, 64, 8, 2, [0, 10, 64, 0, 127], [200, 54, 1, 0, 66], 128, False, False, 7),
    "prompts_block_d64": ("fp8_block", 64, 16, 16, 1, [5, 0, 15], [40, 16, 1], 64, False, True, 1),
    "prompts_bf16_partial": ("bf16", 128, 48, 4, 1, [0, 47, 20], [100, 2, 0], 32, False, False, 2),
    "prompts_bf16_pairs": ("bf16", 64, 32, 6, 6, [33], [77], 48, True, True, 0),
    "prompts_f32": ("f32", 64, 16, 8, 2, [0, 7, 700], [333, 0, 12], 16, True, False, 0),
    "prompts_f32_d128": ("f32", 128, 16, 2, 2, [1], [35], 96, False, False, 0),
    "prompts_g32": ("fp8", 128, 64, 8, 4, [0, 70], [65, 130], 128, False, False, 4),
    "prompts_g32_odd_rotary": ("fp8", 128, 16, 8, 4, [9], [23], 48, False, False, 0),
    "block_of_one": ("fp8_block", 128, 1, 2, 1, [0, 3], [5, 2], 128, False, False, 0),
    "block_of_five": ("fp8_block", 128, 5, 2, 2, [0, 3, 4], [11, 2, 1], 64, False, False, 0),
    "block_of_256": ("fp8_block", 128, 256, 16, 1, [100, 0], [300, 256], 128, True, False, 0),
    "no_rotation": ("fp8_block", 128, 64, 4, 4, [30], [50], 0, False, False, 0),
    "many_requests": ("bf16", 64, 16, 2, 1, [i % 37 for i in range(90)], [i % 5 for i in range(90)], 64, False, False, 11),
    "many_single_rows": ("fp8_block", 64, 16, 2, 1, [i for i in range(70)], [1] * 70, 64, False, True, 2),
    "many_prompts": ("fp8_block", 128, 64, 4, 4, [i % 70 for i in range(45)], [7 * i % 90 for i in range(45)], 128, False, False, 0),
    "many_prompts_d64": ("fp8_block", 64, 100, 4, 4, [i % 70 for i in range(45)], [7 * i % 120 for i in range(45)], 64, False, False, 0),
    "prompts_block_16": ("fp8_block", 128, 16, 4, 2, [0, 5, 16], [40, 30, 9], 128, False, False, 0),
    "prompts_block_32": ("fp8_block", 128, 32, 4, 2, [0, 5, 33], [70, 30, 9], 128, True, False, 0),
    "prompts_g32_256": ("fp8", 64, 256, 4, 2, [0, 5], [300, 30], 64, False, False, 0),
    "long_prompts": ("bf16", 64, 64, 2, 1, [0, 100, 3, 9], [4001, 4102, 77, 1], 64, False, False, 5),
    "long_prompts_block": ("fp8_block", 64, 32, 32, 2, [5, 0, 7], [2000, 2, 2099], 32, True, True, 3),
    "no_new_rows": ("fp8_block", 64, 16, 2, 1, [5, 0], [0, 0], 64, False, False, 3),
}


@pytest.mark.parametrize("name", list(CASES))
def test_append_matches_the_definition(name):
    w = World(*CASES[name], seed=len(name))
    w.append()
    check(w)
    check_summaries(w)
    # the same call again changes nothing: the same rows at the same places
    before = [t.clone() for t in (w.g["k"], w.g["v"], w.q_out, w.smin, w.smax)]
    w.append()
    for a, b in zip(before, (w.g["k"], w.g["v"], w.q_out, w.smin, w.smax)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check(w)


@pytest.mark.parametrize("kind", ["fp8_block", "bf16"])
def test_without_query_and_without_summaries(kind):
    w = World(kind, 128, 16, 4, 2, [20, 0], [30, 3], 128, seed=5)
    w.append(q=False, summaries=False)
    assert (w.q_out == SENTINEL).all()
    lo = w.smin.clone()
    w.append(q=True, summaries=False)
    assert torch.equal(lo, w.smin)
    check(w)


def test_no_rows_at_all():
    """Nothing to append: an empty batch of rows is not an error, and nothing changes."""
    w = World("fp8_block", 64, 16, 4, 2, [5, 20], [0, 0], 64, pad=0, seed=2)
    keep = [t.clone() for t in (w.g["k"], w.gs["k"], w.smin)]
    assert w.kn.shape[0] == 0 and w.params._requests == 2
    w.append()
    assert w.hs.hs_get_device_error() == (w.hs.HS_OK, 0)
    for a, b in zip(keep, (w.g["k"], w.gs["k"], w.smin)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8_block"])
@pytest.mark.parametrize("n", [1, 20])
def test_channels_of_nothing_but_not_a_number(kind, n):
    """Their summary is what the builder gives (no bound at all), and does not spoil what later rows give."""
    w = World(kind, 64, 16, 2, 1, [0], [n], 0, seed=3)
    w.kn[:, :, 5] = float("nan")
    w.append()
    check_summaries(w)
    w.gl += 1
    w.offsets = None
    row = torch.ones((1, 1, 64), dtype=w.wide, device="cuda")
    w.hs.hs_append_tokens(w.shape, w.kv, w.hs.append_params(), row, row, None, None, w.smin, w.smax)
    check_summaries(w)
    assert torch.isfinite(w.smin[0, 0, n // 16]).all()


@pytest.mark.parametrize("d,rotary,interleaved", [(128, 128, False), (128, 64, False), (128, 96, True), (64, 48, False), (64, 0, False)])
@pytest.mark.parametrize("n", [1, 90])
def test_grouped_codes_are_those_of_the_quantiser(d, rotary, interleaved, n):
    """Bit for bit, for rows that are not rotated (V): ordinary ones, zeros, and groups of the smallest and largest sizes."""
    w = World("fp8", d, 16, 4, 2, [0], [n], rotary, interleaved, seed=8, spread=4.0)
    if n > 1:
        w.vn[5] = 0
        w.vn[6, :, :32] *= 1e-30
        w.vn[7] *= 1e36
        w.vn[8, 1] *= 1e-37
        w.vn[9] = torch.exp2(torch.randint(-30, 30, w.vn[9].shape, device="cuda").float()).to(w.wide)
    w.append()
    codes, scales = O.quantize_e4m3_g32(w.vn.float().cpu().numpy().reshape(-1, d))
    codes, scales = codes.reshape(n, w.hkv, d), scales.reshape(n, w.hkv, d // 32)
    for t in range(n):
        for h in range(w.hkv):
            page = w.table[0, h, t // 16]
            assert np.array_equal(w.g["v"][page, t % 16].cpu().numpy(), codes[t, h]), (t, h)
            assert np.array_equal(w.gs["v"][page, t % 16].cpu().numpy(), scales[t, h]), (t, h)


@pytest.mark.parametrize("d,rotary,interleaved", [(128, 128, False), (128, 96, True), (64, 0, False)])
@pytest.mark.parametrize("n", [1, 90])
def test_grouped_codes_keep_the_sign_of_zero(d, rotary, interleaved, n):
    """-0 among other values, groups of nothing but -0, negative values too small for a code: bit for bit the quantiser's
    codes (0x80), by the append of many rows and of one, as by the one-token call."""
    from query_aware_sparse_hs_gb300 import hs
    w = World("fp8", d, 16, 4, 2, [0], [n], rotary, interleaved, seed=8)
    w.vn[:, :, ::3] = -0.0
    w.vn[:, :, 1::6] = 0.0
    w.vn[:, 0, :32] = -0.0
    w.vn[:, 1, 33] = -2.0 ** -130
    w.append()
    codes = torch.empty((n * w.hkv, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n * w.hkv, d // 32), device="cuda")
    hs.hs_quantize_e4m3_g32(w.vn.contiguous(), codes, scales)
    assert (codes.view(n, w.hkv, d)[:, :, 0] == 0x80).all()
    t = torch.arange(n, device="cuda")
    page = w.gt[0, :, t // 16].T.long()  # [n, hkv]
    assert torch.equal(w.g["v"][page, (t % 16)[:, None]], codes.view(n, w.hkv, d))
    assert torch.equal(w.gs["v"][page, (t % 16)[:, None]], scales.view(n, w.hkv, -1))
    # the last token again by the one-token call: the same bytes
    before = w.g["v"].clone()
    hs.hs_append_token(w.shape, w.kv, w.vn[n - 1:].contiguous(), w.vn[n - 1:].contiguous(), w.smin, w.smax)
    assert torch.equal(before, w.g["v"])


def test_grouped_codes_of_every_quotient_of_two_bf16_significands():
    """Every significand of a group's largest value against every one of the others and 24 exponents, either sign: the
    quotients that the append corrects instead of dividing give the quantiser's codes, bit for bit."""
    from query_aware_sparse_hs_gb300 import hs
    d, block = 64, 256
    top = 1 + torch.arange(128, dtype=torch.float64) / 128
    x = (top[None, :] * torch.exp2(-1.0 - torch.arange(24, dtype=torch.float64))[:, None]).flatten()  # below every top
    x = torch.cat([x, -x, x[:(31 - 2 * len(x) % 31) % 31]]).view(-1, 31)
    g = torch.cat([top[:, None, None].expand(128, len(x), 1), x[None].expand(128, -1, -1)], 2).reshape(-1, d)
    for unit in (1.0, 2.0 ** -40, 2.0 ** 70):  # scales inside the corrected range, and past it
        v = (g * unit).to(torch.bfloat16)
        assert torch.equal(v.double(), g * unit)
        v = v.cuda()
        n = len(v)
        pages = torch.zeros((-(-n // block), block, d), dtype=torch.uint8, device="cuda")
        k, ks = torch.zeros_like(pages), torch.zeros(pages.shape[:2] + (2,), device="cuda")
        vs = torch.zeros_like(ks)
        table = torch.arange(len(pages), dtype=torch.int32, device="cuda").view(1, 1, -1)
        lens, off = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
        kv = hs.paged_kv(k, pages, table, lens, ks, vs)
        hs.hs_append_tokens(hs.attn_shape(1, 1, d, block, "fp8"), kv, hs.append_params(new_offsets=off), v[:, None], v[:, None])
        codes, scales = torch.empty((n, d), dtype=torch.uint8, device="cuda"), torch.empty((n, 2), device="cuda")
        hs.hs_quantize_e4m3_g32(v, codes, scales)
        for got_c, got_s in ((pages, vs), (k, ks)):
            assert torch.equal(got_c.view(-1, d)[:n], codes) and torch.equal(got_s.view(-1, 2)[:n], scales)


@pytest.mark.parametrize("kind,new", [("fp8_block", [i % 5 for i in range(2500)]), ("bf16", [0] * 2499 + [70]), ("fp8", [1] * 2500),
                                      ("fp8_block", [1] * 2500), ("f32", [0, 1] * 1250)])
def test_thousands_of_requests(kind, new):
    w = World(kind, 64, 16, 2, 1, [i % 37 for i in range(2500)], new, 32, seed=11)
    w.append()
    check(w)
    check_summaries(w)


def test_query_in_place():
    w = World("bf16", 128, 16, 4, 2, [20, 0], [30, 3], 128, seed=6)
    w.append()
    q = w.q.clone()
    w.hs.hs_append_tokens(w.shape, w.kv, w.params, w.kn, w.vn, q, q, None, None)
    assert torch.equal(q, w.q_out)
    # and within the fused rows themselves
    w.hs.hs_append_tokens(w.shape, w.kv, w.params, w.kn, w.vn, w.q, w.q, None, None)
    assert torch.equal(w.q, w.q_out)


def test_token_by_token_keeps_the_scale_and_the_summary_true():
    """64 appends into one page whose values grow: the scale only doubles up, the codes stay within the sum of the
    roundings, the summary is the builder's after every token."""
    from query_aware_sparse_hs_gb300 import hs
    d, block, n = 128, 64, 64
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((n, 1, d)) * np.exp2(np.linspace(-12, 6, n))[:, None, None]).to(torch.bfloat16).cuda()
    pages = torch.zeros((1, block, d), dtype=torch.uint8, device="cuda")
    scale = {w: torch.full((1,), float("nan"), device="cuda") for w in "kv"}  # a fresh page's scale is not read
    vp = torch.zeros_like(pages)
    table, lens = torch.zeros((1, 1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    shape = hs.attn_shape(1, 1, d, block, "fp8_block")
    kv = hs.paged_kv(pages, vp, table, lens, scale["k"], scale["v"])
    smin = torch.full((1, 1, 1, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    smax = smin.clone()
    last = 0.0
    for i in range(n):
        lens.fill_(i + 1)
        if i % 2:
            hs.hs_append_token(shape, kv, x[i:i + 1], x[i:i + 1], smin, smax)  # the same by the one-token call
        else:
            hs.hs_append_tokens(shape, kv, hs.append_params(), x[i:i + 1], x[i:i + 1], None, None, smin, smax)
        s = float(scale["k"])
        assert s >= last and s == power_scale(float(x[:i + 1].abs().max())) and float(scale["v"]) == s
        last = s
        lo, hi = torch.full_like(smin, SENTINEL), torch.full_like(smax, SENTINEL)
        hs.hs_build_block_summaries(shape, kv, 0, lo, hi)
        assert torch.equal(smin, lo) and torch.equal(smax, hi), i
    held = O.e4m3_decode(pages[0].cpu().numpy()) * last
    want = x[:, 0].double().cpu().numpy()
    # one rounding of the value (2^-4 of it), and under the smallest normal half a step at each scale: 2^-10 (s + s/2 + ...)
    assert (np.abs(held - want) <= 2.0 ** -4 * np.abs(want) + 2 * 2.0 ** -10 * last).all()
    assert torch.equal(pages, vp)


def test_values_that_are_not_finite_and_pages_of_zeros():
    from query_aware_sparse_hs_gb300 import hs
    d, block = 64, 16
    x = torch.randn((4, 1, d), device="cuda", dtype=torch.bfloat16)
    x[0, 0, 3], x[1, 0, 4], x[2, 0, 5] = float("inf"), float("-inf"), float("nan")
    zero = torch.zeros_like(x)
    table = torch.tensor([[[1, 0]]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([4], dtype=torch.int32, device="cuda")
    k, v = torch.zeros((2, block, d), dtype=torch.uint8, device="cuda"), torch.zeros((2, block, d), dtype=torch.uint8, device="cuda")
    ks, vs = torch.full((2,), float("nan"), device="cuda"), torch.full((2,), float("nan"), device="cuda")
    shape = hs.attn_shape(1, 1, d, block, "fp8_block")
    kv = hs.paged_kv(k, v, table, lens, ks, vs)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    hs.hs_append_tokens(shape, kv, hs.append_params(new_offsets=off), x, zero)
    fin = x[torch.isfinite(x)].abs().max()
    assert float(ks[1]) == power_scale(float(fin)) and float(vs[1]) == 2.0 ** -117 and torch.isnan(ks[0])
    got = O.e4m3_decode(k[1].cpu().numpy())
    assert got[0, 3] == 448 and got[1, 4] == -448 and np.isnan(got[2, 5])
    assert np.array_equal(np.delete(k[1, :4].cpu().numpy().ravel(), 2 * d + 5),
                          np.delete(O.e4m3_encode((x[:, 0].float() / ks[1]).cpu().numpy()).ravel(), 2 * d + 5))
    assert (v == 0).all()
    # a later row gives the page of zeros a scale
    lens.fill_(5)
    hs.hs_append_tokens(shape, kv, hs.append_params(), x[3:], x[3:])
    assert float(vs[1]) == power_scale(float(x[3].abs().max())) and (v[1, :4] == 0).all() and (v[1, 4] != 0).any()
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)


@pytest.mark.parametrize("d,block,batch", [(128, 16, 2), (128, 64, 2), (128, 64, 45), (64, 32, 3), (64, 256, 2), (128, 5, 2)])
def test_infinities_in_pages_of_any_size(d, block, batch):
    """The scale goes by the page's finite values, whether its rows are held or read once more."""
    new = [1 + (37 * i + 90) % 130 for i in range(batch)]
    w = World("fp8_block", d, block, 4, 4, [0] * batch, new, d, seed=9)
    rng = np.random.default_rng(9)
    for row in rng.choice(w.rows, max(3, w.rows // 40), replace=False):
        w.vn[row, rng.integers(4), rng.integers(d)] = float("inf") if row % 2 else float("-inf")
    w.append(q=False)
    assert w.hs.hs_get_device_error() == (w.hs.HS_OK, 0)
    v, codes, scales = w.vn.float().cpu().numpy(), w.g["v"].cpu().numpy(), w.gs["v"].cpu().numpy()
    for b in range(batch):
        o = int(w.offsets[b])
        for j in range(-(-new[b] // block)):
            for h in range(4):
                x = v[o + j * block:min(o + (j + 1) * block, o + new[b]), h]
                page = w.table[b, h, j]
                assert scales[page] == power_scale(float(np.abs(x[np.isfinite(x)]).max()))
                assert np.array_equal(codes[page, :len(x)], O.e4m3_encode(x / scales[page]))


def test_bad_pages_lengths_offsets_and_positions_are_reported_and_skipped():
    w = World("fp8_block", 128, 16, 4, 1, [20, 0, 5], [30, 20, 3], 128, pad=2, seed=9)
    hs = w.hs
    keep = {x: w.g[x].clone() for x in "kv"}
    # request 0: its block 2 has no page; request 1: a page id past the pool in block 1
    w.gt[0, 0, 2] = -1
    w.gt[1, 0, 1] = w.pages
    w.append()
    assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, hs.HS_EBIT_PAGE_RANGE)
    assert not torch.equal(w.g["k"][w.table[1, 0, 0]], keep["k"][w.table[1, 0, 0]])  # its block 0 was written
    assert torch.equal(w.g["k"][w.table[1, 0, 1]], keep["k"][w.table[1, 0, 1]])
    assert torch.equal(w.g["v"][w.table[0, 0, 2]], keep["v"][w.table[0, 0, 2]])
    assert (w.smin[0, 0, 2] == SENTINEL).all()

    # more new rows than tokens; a request past the page table; positions past the angles
    w = World("fp8_block", 128, 16, 4, 1, [20, 0, 5], [30, 20, 3], 128, pad=2, seed=9)
    keep = {x: w.g[x].clone() for x in "kv"}
    w.gl[0] = 29
    w.gl[1] = w.mb * 16 + 4
    w.append()
    assert hs.hs_get_device_error()[0] == hs.HS_ERR_OUT_OF_RANGE
    assert torch.equal(w.g["k"][w.table[0, 0, :4]], keep["k"][w.table[0, 0, :4]])
    assert not torch.equal(w.g["k"][w.table[2, 0, 0]], keep["k"][w.table[2, 0, 0]])
    assert (w.q_out[:30] == SENTINEL).all() and (w.q_out[50:53] != SENTINEL).any()

    w = World("bf16", 128, 16, 4, 1, [20, 0, 5], [30, 20, 3], 128, positions=True, pad=2, seed=9)
    keep = {x: w.g[x].clone() for x in "kv"}
    bad = w.params._keep[2]
    bad[51], bad[30] = w.params.table_rows, -1  # rows 1 of request 2 and 0 of request 1
    w.append()
    assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, hs.HS_EBIT_POSITION)
    page = int(w.table[2, 0, 0])
    assert torch.equal(w.g["k"][page, 6], keep["k"][page, 6]) and not torch.equal(w.g["v"][page, 6], keep["v"][page, 6])
    assert not torch.equal(w.g["k"][page, 5], keep["k"][page, 5])
    assert (w.q_out[51] == SENTINEL).all() and (w.q_out[30] == SENTINEL).all() and (w.q_out[52] != SENTINEL).any()

    # offsets that descend, or pass the rows: nothing out of range is read or written
    for o in ([0, 40, 20, 53], [0, 30, 50, 4000], [-5, 30, 50, 53], [7, 3, 1, 0]):
        w = World("fp8_block", 128, 16, 4, 1, [20, 0, 5], [30, 20, 3], 128, pad=2, seed=9)
        w.params._keep[1].copy_(torch.tensor(o, dtype=torch.int32))
        w.append()
        torch.cuda.synchronize()
        hs.hs_get_device_error()


ONE_ROW = {
    # as CASES, one new token per request and no offsets: kind, d, block, hq, hkv, earlier tokens, rotary, interleaved, positions
    "f32": ("f32", 64, 16, 8, 2, [0, 5, 16, 31], 64, False, True),
    "f32_partial": ("f32", 128, 16, 4, 4, [0, 15, 47], 96, False, False),
    "f32_pairs": ("f32", 128, 5, 2, 1, [4, 5, 6], 128, True, False),
    "f32_unrotated": ("f32", 64, 16, 2, 2, [3, 0], 0, False, False),
    "bf16_positions": ("bf16", 128, 64, 32, 4, [0, 63, 64, 1], 128, False, True),
    "bf16_pairs": ("bf16", 64, 32, 6, 6, [0, 33], 48, True, True),
    "bf16_one_head": ("bf16", 64, 16, 1, 1, [9], 16, False, False),
    "g32_positions": ("fp8", 128, 16, 8, 8, [0, 16, 17], 128, False, True),
    "g32_partial": ("fp8", 128, 16, 4, 2, [3, 20], 48, False, False),
    "g32_pairs": ("fp8", 128, 48, 2, 2, [47, 48], 96, True, False),
    "block_positions": ("fp8_block", 128, 64, 32, 4, [0, 63, 64, 130, 1], 128, False, True),
    "block_partial": ("fp8_block", 128, 256, 4, 2, [255, 256, 100], 32, False, False),
    "block_pairs": ("fp8_block", 64, 16, 16, 1, [5, 16, 0], 64, True, True),
    "block_pairs_d128": ("fp8_block", 128, 5, 2, 2, [3, 4, 5, 44], 96, True, False),
    "block_of_one": ("fp8_block", 64, 1, 2, 1, [0, 3], 64, False, False),
    "block_unrotated": ("fp8_block", 128, 48, 4, 4, [30, 0], 0, False, False),
}


def one_row_world(name, grow=0, **kw):
    kind, d, block, hq, hkv, old, rotary, interleaved, positions = ONE_ROW[name]
    w = World(kind, d, block, hq, hkv, old, [1] * len(old), rotary, interleaved, positions, seed=len(name), **kw)
    assert w.offsets is None
    if grow:
        w.kn *= 2.0 ** grow
        w.vn *= 2.0 ** grow
        w.qkv[:, hq:] *= 2.0 ** grow
    return w


@pytest.mark.parametrize("grow", [0, 7, -12])
@pytest.mark.parametrize("name", list(ONE_ROW))
def test_one_row_per_request_matches_the_definition(name, grow):
    """Rows of the size of the earlier ones, larger (a page's scale has to grow: the earlier codes and their summary are
    taken anew, whichever channels the rotation gave a thread) and smaller."""
    w = one_row_world(name, grow)
    before = {x: None if w.gs[x] is None else w.gs[x].clone() for x in "kv"}
    w.append()
    check(w)
    check_summaries(w)
    if grow > 0 and w.kind == "fp8_block":
        last = [w.table[b, :, n // w.block] for b, n in enumerate(w.old) if n % w.block]
        if last:
            pages = torch.from_numpy(np.concatenate(last)).long().cuda()
            assert (w.gs["k"][pages] > before["k"][pages]).all() and (w.gs["v"][pages] > before["v"][pages]).all()
    keep = [t.clone() for t in (w.g["k"], w.g["v"], w.q_out, w.smin, w.smax)]
    w.append()
    for a, b in zip(keep, (w.g["k"], w.g["v"], w.q_out, w.smin, w.smax)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name", ["f32", "bf16_positions", "g32_positions", "block_positions", "block_pairs"])
def test_one_row_per_request_reports_and_skips_what_is_out_of_range(name):
    def of(w, b):  # what request b's append may write
        pages = torch.from_numpy(w.table[b][w.table[b] >= 0]).long().cuda()
        return [t[pages] for t in (w.g["k"], w.g["v"])] + [w.smin[b], w.smax[b]] + [t[pages] for t in (w.gs["k"], w.gs["v"]) if t is not None]

    def same(a, b):
        return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))

    good = one_row_world(name)
    good.append()
    hs, last = good.hs, len(good.new) - 1

    def others(w):  # the other requests are as in the good call
        assert all(same(of(w, b), of(good, b)) and torch.equal(w.q_out[b], good.q_out[b]) for b in range(last + 1) if b != 1)

    # no token: nothing is written for the request, and nothing is wrong with that
    w = one_row_world(name)
    was = of(w, 1)
    w.gl[1] = 0
    w.append()
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    assert same(of(w, 1), was) and (w.q_out[1] == SENTINEL).all()
    others(w)
    # no page, a page past the pool, a block past the table: Q needs none of them
    for change, bit in (("gt", hs.HS_EBIT_PAGE_RANGE), ("pool", hs.HS_EBIT_PAGE_RANGE), ("gl", hs.HS_EBIT_BLOCK_RANGE)):
        w = one_row_world(name)
        was, j = of(w, 1), w.old[1] // w.block
        if change == "gl":
            w.gl[1] = w.mb * w.block + 1
            w.params = hs.append_params(w.params._keep[0], w.interleaved, None, torch.zeros(last + 1, dtype=torch.int32, device="cuda"))
        else:
            w.gt[1, :, j] = -1 if change == "gt" else w.pages
        w.append()
        assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, bit), change
        assert same(of(w, 1), was)
        if change != "gl":
            others(w)
    # a position without angles: K, its summary and scale and Q stay, V is written
    for bad in (-1, w.cos_sin.shape[0], 2 ** 31 - 1):
        w = one_row_world(name)
        was = of(w, 1)
        w.params._keep[2][1] = bad
        w.append()
        assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, hs.HS_EBIT_POSITION)
        now, want = of(w, 1), of(good, 1)
        assert same([now[0]] + now[2:5], [was[0]] + was[2:5])
        assert same([now[1]] + now[5:], [want[1]] + want[5:]) and (w.q_out[1] == SENTINEL).all()
        others(w)


OFFSETS = {
    # block, earlier tokens, rows of each request, offsets given instead
    "descend": (16, [20, 0, 5], [30, 20, 3], [0, 40, 20, 53]),
    "past_the_rows": (16, [20, 0, 5], [30, 20, 3], [0, 30, 50, 4000]),
    "negative": (16, [20, 0, 5], [30, 20, 3], [-5, 30, 50, 53]),
    "all_descend": (16, [20, 0, 5], [30, 20, 3], [7, 3, 1, 0]),
    "one_hidden_by_the_others": (16, [20, 0, 57], [30, 20, 3], [0, 32, 0, 53]),  # two blocks back: the next request's slots
    "one_hidden_64": (64, [20, 0, 170], [150, 20, 3], [0, 128, 0, 173]),
    "one_hidden_blocks_of_one": (1, [3, 0, 5], [5, 2, 4], [0, 5, 3, 9]),
    "extremes": (16, [20, 0, 5], [30, 20, 3], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 53]),
    "many": (16, [i % 37 for i in range(90)], [2 + i % 5 for i in range(90)], {41: 0}),
    "many_last": (16, [i % 37 for i in range(90)], [2 + i % 5 for i in range(90)], {90: 100000}),
}


@pytest.mark.parametrize("name", list(OFFSETS))
@pytest.mark.parametrize("kind", ["fp8_block", "bf16"])
def test_every_request_whose_offsets_do_not_ascend_is_reported(name, kind):
    """The error bit, whatever the other requests' offsets are; the bad requests' pages, scales and summaries stay as they
    were, the others are written (but for those that a descent hides)."""
    block, old, new, given = OFFSETS[name]
    w = World(kind, 64, block, 4, 2, old, new, 64, pad=2, seed=9)
    hs, n = w.hs, len(new)
    o = w.offsets.tolist()
    o = [given.get(i, x) for i, x in enumerate(o)] if isinstance(given, dict) else given
    w.params._keep[1].copy_(torch.tensor(o, dtype=torch.int32))
    bad = [o[b] < 0 or o[b + 1] < o[b] or o[b + 1] > w.rows or o[b + 1] - o[b] > w.lens[b] for b in range(n)]
    keep = {x: w.g[x].clone() for x in "kv"}, {x: None if w.gs[x] is None else w.gs[x].clone() for x in "kv"}, w.smin.clone()
    assert any(bad)
    w.append()
    assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, hs.HS_EBIT_BLOCK_RANGE)
    for b in range(n):
        pages = torch.from_numpy(w.table[b][w.table[b] >= 0]).long().cuda()
        for x in "kv":
            same = torch.equal(w.g[x][pages].view(torch.uint8), keep[0][x][pages].view(torch.uint8))
            assert same or not bad[b], (b, x)
            assert not same or bad[b] or o[b] == o[b + 1] or name == "many", (b, x)
            if bad[b] and w.gs[x] is not None:
                assert torch.equal(w.gs[x][pages], keep[1][x][pages])
        if bad[b]:
            assert torch.equal(w.smin[b], keep[2][b])


def test_offsets_are_checked_where_there_are_no_rows():
    w = World("bf16", 64, 16, 4, 2, [5, 20], [0, 0], 64, seed=2)
    keep = w.g["k"].clone()
    w.params._keep[1].copy_(torch.tensor([0, 0, 5], dtype=torch.int32))
    w.append()
    assert w.hs.hs_get_device_error() == (w.hs.HS_ERR_OUT_OF_RANGE, w.hs.HS_EBIT_BLOCK_RANGE)
    assert torch.equal(keep, w.g["k"])


def test_tables_that_are_not_on_the_gpu_are_refused():
    w = World("bf16", 64, 16, 4, 2, [5, 20], [3, 4], 64, positions=True, seed=2)
    cos_sin, off, pos = w.params._keep[0], w.params._keep[1], w.params._keep[2]
    keep = w.g["k"].clone()
    with pytest.raises(ValueError):
        w.hs.append_params(cos_sin, new_offsets=off.cpu(), positions=pos)
    for p in (w.hs.append_params(cos_sin.cpu(), new_offsets=off.cpu()), w.hs.append_params(new_offsets=off.cpu())):
        with pytest.raises(ValueError, match="on the current device"):
            w.hs.hs_append_tokens(w.shape, w.kv, p, w.kn, w.vn)
    assert torch.equal(keep, w.g["k"])


def test_other_streams_and_graphs():
    a, b = (World(*CASES["prompts_block"], seed=4) for _ in range(2))
    a.append()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.append()
    side.synchronize()
    for x, y in ((a.g["k"], b.g["k"]), (a.g["v"], b.g["v"]), (a.q_out, b.q_out), (a.smin, b.smin)):
        assert torch.equal(x, y)
    # captured once, replayed as the requests grow
    w = World("fp8_block", 128, 16, 4, 2, [20, 3], [1, 1], 128, seed=8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.append()
    graph.replay()
    check(w)
    check_summaries(w)
