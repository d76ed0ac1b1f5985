"""Attention weights accumulated per token, and the eviction of the lightest tokens, over caches of every kind, against plain
64-bit arithmetic; decode, accumulate, evict and decode again as one run.  GPU only."""

import numpy as np
import pytest
import torch

import _int4
import oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
KINDS = ["f32", "bf16", "fp8", "fp8_block", "int4"]


class Cache:
    """A paged cache of any kind with random values, rows of nobody poisoned; `rows` gives 64-bit values."""

    def __init__(self, kind, lens, hkv, d, block, seed=0, spare=2, mb=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.kind, self.lens, self.hkv, self.d, self.block, self.rng = kind, list(lens), hkv, d, block, rng
        self.nb = [-(-n // block) for n in lens]
        self.mb = mb or max(1, max(self.nb)) + 1
        pages = sum(self.nb) * hkv + spare
        order = rng.permutation(pages)
        self.table = np.full((len(lens), hkv, self.mb), -1, np.int32)
        at = 0
        for b, n in enumerate(self.nb):
            for h in range(hkv):
                self.table[b, h, :n] = order[at:at + n]
                at += n
        shape = (pages, block, d)
        self.x, self.sc = {}, {"k": None, "v": None}
        for w in "kv":
            if kind in ("f32", "bf16"):
                self.x[w] = torch.randn(shape, generator=g).to(torch.float32 if kind == "f32" else torch.bfloat16)
            elif kind == "int4":
                self.x[w] = torch.randint(0, 256, shape[:2] + (d // 2,), generator=g, dtype=torch.uint8)
                s = 0.1 + 0.3 * torch.rand(shape[:2] + (1, d // 32), generator=g)
                self.sc[w] = torch.cat([s, 0.4 * torch.randn(s.shape, generator=g)], 2).to(torch.bfloat16)
            else:
                self.x[w] = torch.from_numpy(O.e4m3_encode(rng.standard_normal(shape) * 90))
                self.sc[w] = 0.004 + 0.01 * torch.rand((pages,) if kind == "fp8_block" else shape[:2] + (d // 32,), generator=g)
        nan = {"f32": np.nan, "bf16": np.nan}.get(kind, 0xFF)  # rows of nobody
        for b, L in enumerate(lens):
            if L % block:
                for h in range(hkv):
                    for w in "kv":
                        p = self.table[b, h, L // block]
                        self.x[w][p, L % block:] = nan
                        if kind in ("int4", "fp8"):
                            self.sc[w][p, L % block:] = np.nan
        for w in "kv":
            self.x[w] = self.x[w].cuda()
            self.sc[w] = None if self.sc[w] is None else self.sc[w].cuda()
        self.gt, self.gl = torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.up()

    def up(self):
        from query_aware_sparse_hs_gb300 import hs
        self.kv = hs.paged_kv(self.x["k"], self.x["v"], self.gt, self.gl, self.sc["k"], self.sc["v"])

    def rows(self, w, b, h, tokens):
        t = np.asarray(tokens, np.int64)
        p, r = torch.from_numpy(self.table[b, h, t // self.block].astype(np.int64)).cuda(), torch.from_numpy(t % self.block).cuda()
        x = self.x[w][p, r]
        if self.kind == "int4":
            return _int4.values(x.cpu().numpy(), self.sc[w][p, r].double().cpu().numpy())
        if self.kind in ("f32", "bf16"):
            return x.double().cpu().numpy()
        s = self.sc[w][p].double().cpu().numpy()[:, None] if self.kind == "fp8_block" else \
            self.sc[w][p, r].double().cpu().numpy().repeat(32, -1)
        return O.e4m3_decode(x.cpu().numpy()) * s

    def shape(self, group):
        from query_aware_sparse_hs_gb300 import hs
        return hs.attn_shape(group * self.hkv, self.hkv, self.d, self.block, self.kind)


def queries(c, group, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((len(c.lens), group * c.hkv, c.d), generator=g).to(torch.float32 if c.kind == "f32" else torch.bfloat16).cuda()


def lse_of(c, q, group, sel, cnt, scale):
    """64-bit log-sum-exp of every head over its selection, as f32."""
    out = np.full(q.shape[:2], -np.inf)
    for b in range(len(c.lens)):
        for h in range(c.hkv):
            t = tokens_of(c, b, sel[b, h, :cnt[b, h]])
            if len(t):
                z = q[b, h * group:(h + 1) * group].double().cpu().numpy() @ c.rows("k", b, h, t).T * scale
                m = z.max(1)
                out[b, h * group:(h + 1) * group] = m + np.log(np.exp(z - m[:, None]).sum(1))
    return torch.from_numpy(out).float().cuda()


def tokens_of(c, b, blocks):
    return np.concatenate([np.zeros(0, np.int64)] + [np.arange(j * c.block, min(c.lens[b], (j + 1) * c.block)) for j in blocks])


def check_weights(c, q, group, lse, sel, cnt, scale, start, got):
    """A logit is off by D fp32 roundings of the magnitudes' sum (grouped and 4-bit scales are applied to partial sums, 4-bit
    codes count as up to 24 scales), its exponential by that and two roundings more, and the sums by one for each head and one
    for the sum with what was there.  8-bit kinds hold a query's entries to 2^-33 of the largest."""
    start, got, ln = start.double().cpu().numpy(), got.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(c.lens)):
        for h in range(c.hkv):
            want = start[b, h].copy()
            err = np.zeros_like(want)
            qn = q[b, h * group:(h + 1) * group].double().cpu().numpy()
            for j in sel[b, h, :cnt[b, h]]:
                t = tokens_of(c, b, [j])
                K = c.rows("k", b, h, t)
                mag = np.abs(K) + (12.0 if c.kind == "int4" else 0.0)
                ds = (mag @ np.abs(qn).T * U * (c.d + 24) + np.abs(K).sum(1)[:, None] * np.abs(qn).max(1) * 2.0 ** -33) * abs(scale)
                live = np.isfinite(ln[b, h * group:(h + 1) * group])
                z = K @ qn.T * scale - np.where(live, ln[b, h * group:(h + 1) * group], 0.0)
                e = np.where(live, np.exp(z), 0.0)
                want[t] += e.sum(1)
                err[t] += (e * (np.expm1(2 * ds + 2 * U * (np.abs(z) + 40)) + 8 * U)).sum(1)
            bound = err + (group + 4) * U * np.abs(want)
            assert (np.abs(got[b, h] - want) <= bound).all(), (b, h, np.abs(got[b, h] - want).max())
            assert (got[b, h][want == start[b, h]] == start[b, h][want == start[b, h]]).all()


CASES = {
    # request lengths, kv heads, group, d, block, blocks kept (None: all)
    "one_token": ([1], 1, 8, 128, 64, None),
    "around_a_tile": ([31, 32, 33, 63, 64, 65], 2, 8, 128, 64, None),
    "pages_of_16_selected": ([900, 30, 2000], 2, 4, 128, 16, 7),
    "pages_of_one": ([5, 40], 1, 2, 128, 1, None),
    "pages_of_five": ([3, 44, 201], 2, 1, 128, 5, None),
    "pages_of_48_group_16": ([48, 47, 700], 1, 16, 128, 48, None),
    "pages_of_256": ([255, 257, 1024], 1, 8, 128, 256, None),
    "d64": ([700, 3, 65], 2, 8, 64, 64, None),
    "d64_group_16": ([333, 1, 64], 1, 16, 64, 16, None),
    "empty_requests": ([0, 100, 0, 0, 5, 0], 2, 8, 128, 16, None),
    "nothing_selected": ([100, 200], 2, 8, 128, 16, 0),
    "one_long_among_short": ([9000] + [3] * 20, 1, 8, 128, 64, None),
    "many_requests": ([1 + 7 * i % 90 for i in range(300)], 2, 2, 64, 16, None),
}


def selection(c, keep, shuffle=False):
    return _int4.chosen(c, max(1, max(c.nb)) if keep is None else max(1, keep), keep, shuffle)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", list(CASES))
def test_weights_are_the_softmax_weights_added_up(kind, name):
    from query_aware_sparse_hs_gb300 import hs
    lens, hkv, group, d, block, keep = CASES[name]
    c = Cache(kind, lens, hkv, d, block, seed=len(name))
    q = queries(c, group)
    sel, cnt = selection(c, keep, shuffle="selected" in name)
    scale = d ** -0.5
    lse = lse_of(c, q, group, sel, cnt, scale)
    start = torch.rand((len(lens), hkv, c.mb * block), generator=torch.Generator().manual_seed(3)).cuda()
    got = start.clone()
    hs.hs_accumulate_attn_weights(c.shape(group), c.kv, q, lse, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(),
                                  sel.shape[2], scale, got)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    check_weights(c, q, group, lse, sel, cnt, scale, start, got)


@pytest.mark.parametrize("kind", KINDS)
def test_weights_of_any_order_twice_selected_negative_scales_and_empty_heads(kind):
    from query_aware_sparse_hs_gb300 import hs
    c = Cache(kind, [300, 90], 2, 128, 16, seed=2)
    q = queries(c, 4)
    sel = np.full((2, 2, 9), -1, np.int32)
    sel[0, 0, :5], sel[0, 1, :2], sel[1, 0, :6] = [18, 3, 3, 0, 7], [1, 0], [5, 4, 3, 2, 1, 0]
    cnt = np.array([[5, 2], [6, 0]], np.int32)
    for scale in (-0.1, 0.0, 0.3):
        lse = lse_of(c, q, 4, sel, cnt, scale)
        lse[0, 1] = -np.inf
        start = torch.zeros((2, 2, c.mb * 16), device="cuda")
        got = start.clone()
        for _ in range(2):
            start = got.clone()
            hs.hs_accumulate_attn_weights(c.shape(4), c.kv, q, lse, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(), 9,
                                          scale, got)
            check_weights(c, q, 4, lse, sel, cnt, scale, start, got)
    # v_pages are not looked at, and results do not depend on the order of arrival
    one = hs.paged_kv(c.x["k"], None, c.gt, c.gl, c.sc["k"], None)
    first = None
    for _ in range(10):
        got = torch.zeros_like(start)
        hs.hs_accumulate_attn_weights(c.shape(4), one, q, lse, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(), 9, scale, got)
        first = got if first is None else first
        assert torch.equal(got, first)


@pytest.mark.parametrize("group", [1, 4, 16])
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_weights_of_tokens_infinitely_far_off(kind, group):
    """A logit of -inf is a weight of 0, whatever the product's places without a head make of an infinite K."""
    from query_aware_sparse_hs_gb300 import hs
    c = Cache(kind, [70, 200], 1, 128, 16)
    q = queries(c, group)
    q[:, :, 32:64] = -q[:, :, 32:64].abs()
    far = {0: [3, 69], 1: [0, 31, 150]}
    sel, cnt = selection(c, None)
    lse = lse_of(c, q, group, sel, cnt, 0.09)  # (of other keys: any will do)
    start = torch.zeros((2, 1, c.mb * 16), device="cuda")

    def run():
        got = start.clone()
        hs.hs_accumulate_attn_weights(c.shape(group), c.kv, q, lse, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(),
                                      sel.shape[2], 0.09, got)
        assert hs.hs_get_device_error() == (hs.HS_OK, 0)
        return got

    want = run()
    for b, tokens in far.items():
        for t in tokens:
            p = int(c.table[b, 0, t // 16])
            if kind == "fp8":
                c.x["k"][p, t % 16, 32:64] = 0x38  # 1.0
                c.sc["k"][p, t % 16, 1] = float("inf")
            else:
                c.x["k"][p, t % 16, 40] = float("inf")
            want[b, 0, t] = 0.0
    assert torch.equal(run(), want)


@pytest.mark.parametrize("kind", KINDS)
def test_weights_report_what_is_out_of_range(kind):
    from query_aware_sparse_hs_gb300 import hs
    c = Cache(kind, [300, 100], 1, 64, 16, seed=9)
    q = queries(c, 8)
    sel = np.full((2, 1, 4), -1, np.int32)
    sel[0, 0], sel[1, 0, :2] = [0, 5, 19, 18], [-2147483648, 3]
    fine, fine_cnt = np.full((2, 1, 4), -1, np.int32), np.array([[3], [1]], np.int32)
    fine[0, 0, :3], fine[1, 0, 0] = [0, 5, 18], 3
    lse = lse_of(c, q, 8, fine, fine_cnt, 0.125)
    zero = torch.zeros((2, 1, c.mb * 16), device="cuda")
    got = zero.clone()
    hs.hs_accumulate_attn_weights(c.shape(8), c.kv, q, lse, torch.from_numpy(sel).cuda(),
                                  torch.tensor([[9], [2]], dtype=torch.int32).cuda(), 4, 0.125, got)
    assert hs.hs_get_device_error()[1] == hs.HS_EBIT_CAPACITY | hs.HS_EBIT_BLOCK_RANGE
    check_weights(c, q, 8, lse, fine, fine_cnt, 0.125, zero, got)
    c.gt[0, 0, 5] = c.x["k"].shape[0]
    got = zero.clone()
    hs.hs_accumulate_attn_weights(c.shape(8), c.kv, q, lse, torch.from_numpy(fine).cuda(), torch.from_numpy(fine_cnt).cuda(), 4,
                                  0.125, got)
    assert hs.hs_get_device_error()[1] == hs.HS_EBIT_PAGE_RANGE
    fine[0, 0, :3], fine_cnt[0] = [0, 18, -1], 2
    check_weights(c, q, 8, lse, fine, fine_cnt, 0.125, zero, got)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_every_head_adds_one(kind):
    """With the lse that the library's attention left, over a long cache."""
    from query_aware_sparse_hs_gb300 import hs
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    c = Cache(kind, [20000, 700], 2, 128, 64, seed=4)
    dec = SparseDecode(num_q_heads=16, num_kv_heads=2, head_dim=128, block_size=64, kv_dtype=kind, batch=2, max_blocks=c.mb,
                       sink_tokens=4, window_tokens=64, k_scored=40)
    q = queries(c, 8)
    dec.build_summaries(c.kv)
    dec.step(c.kv, q)
    w = torch.zeros((2, 2, c.mb * 64), device="cuda")
    dec.accumulate_weights(c.kv, q, w)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    assert (w.sum(-1) - 8).abs().max() < 8 * 1e-4 and (w >= 0).all()
    with pytest.raises(ValueError):
        other = SparseDecode(num_q_heads=16, num_kv_heads=2, head_dim=128, block_size=64, kv_dtype=kind, batch=2,
                             max_blocks=c.mb, sink_tokens=4, window_tokens=64, k_scored=9)
        dec.accumulate_weights(c.kv, q, w, selection=other)


# ---- eviction ------------------------------------------------------------------------------------------------------------


def kept_of(w, L, budget, sink, recent):
    """Which tokens stay, from the definition."""
    if L <= budget:
        return np.arange(L)
    free = np.arange(sink, L - recent)
    x = np.where(np.isnan(w[free]), -np.inf, w[free] + 0.0)
    nan = np.isnan(w[free])
    order = sorted(range(len(free)), key=lambda i: (nan[i], -x[i], i))[:budget - sink - recent]
    return np.sort(np.concatenate([np.arange(sink), free[np.array(order, int)], np.arange(L - recent, L)]))


def destination(c, budget, seed=7, spare=3, mb=None):
    """An empty cache with room for `budget` tokens a request: pages, scales, table, lengths, weights."""
    from query_aware_sparse_hs_gb300 import hs
    nb = [-(-min(L, budget) // c.block) for L in c.lens]
    mb = mb or -(-budget // c.block) + 1
    pages = sum(nb) * c.hkv + spare
    order = np.random.default_rng(seed).permutation(pages)
    table = np.full((len(c.lens), c.hkv, mb), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        for h in range(c.hkv):
            table[b, h, :n] = order[at:at + n]
            at += n
    x = {w: torch.full((pages,) + c.x[w].shape[1:], 9, dtype=c.x[w].dtype, device="cuda") for w in "kv"}
    sc = {w: None if c.sc[w] is None else torch.full((pages,) + c.sc[w].shape[1:], 9, dtype=c.sc[w].dtype, device="cuda") for w in "kv"}
    lens = torch.full((len(c.lens),), -5, dtype=torch.int32, device="cuda")
    gt = torch.from_numpy(table).cuda()
    return {"x": x, "sc": sc, "table": table, "lens": lens, "w": torch.full((len(c.lens), c.hkv, mb * c.block), 9.0, device="cuda"),
            "kv": hs.paged_kv(x["k"], x["v"], gt, lens, sc["k"], sc["v"]), "gt": gt}


def check_evicted(c, d, w, budget, sink, recent, kept, with_weights=True):
    wn = w.cpu().numpy()
    kn, dw = kept.cpu().numpy(), d["w"].cpu().numpy()
    assert d["lens"].tolist() == [min(L, budget) for L in c.lens]
    left = {k: torch.ones(x.shape[:2], dtype=torch.bool) for k, x in d["x"].items()}
    for b, L in enumerate(c.lens):
        for h in range(c.hkv):
            t = kept_of(wn[b, h], L, budget, sink, recent)
            assert kn[b, h].tolist() == t.tolist() + [-1] * (budget - len(t)), (b, h)
            i = np.arange(len(t))
            if with_weights:
                assert np.array_equal(dw[b, h, :len(t)], wn[b, h, t], equal_nan=True) and (dw[b, h, len(t):] == 9).all()
            src = torch.from_numpy(c.table[b, h, t // c.block].astype(np.int64)).cuda(), torch.from_numpy(t % c.block).cuda()
            dst = torch.from_numpy(d["table"][b, h, i // c.block].astype(np.int64)).cuda(), torch.from_numpy(i % c.block).cuda()
            for k in "kv":
                a, z = c.x[k][src], d["x"][k][dst]
                assert torch.equal(a.view(torch.uint8), z.view(torch.uint8)), (k, b, h)
                if c.sc[k] is not None:
                    assert torch.equal(c.sc[k][src], d["sc"][k][dst])
                left[k][d["table"][b, h, i // c.block], i % c.block] = False
    for k in "kv":  # rows of nobody
        assert (d["x"][k].float()[left[k].cuda()] == 9).all()


def weights_for(c, seed=11, ties=True):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand((len(c.lens), c.hkv, c.mb * c.block), generator=g) ** 6
    if ties:
        w = torch.where(torch.rand(w.shape, generator=g) < 0.4, (w * 8).round() / 8, w)
    return w.cuda()


EVICTS = {
    # request lengths, kv heads, d, block, budget, sink, recent
    "ordinary": ([3000, 700, 64, 65], 2, 128, 64, 256, 4, 64),
    "budget_of_one": ([100, 1, 0], 2, 128, 16, 1, 0, 0),
    "one_of_sink": ([100, 1, 0], 1, 64, 16, 1, 1, 0),
    "one_recent": ([100, 1, 0], 1, 64, 16, 1, 0, 1),
    "only_sink_and_recent": ([500, 30], 2, 128, 16, 40, 10, 30),
    "exactly_the_budget": ([128, 129, 127], 2, 64, 32, 128, 4, 32),
    "no_sink_no_recent": ([2000, 37], 1, 128, 48, 333, 0, 0),
    "pages_of_five": ([201, 44, 3], 2, 64, 5, 33, 2, 7),
    "pages_of_one": ([90, 5], 1, 128, 1, 17, 1, 3),
    "pages_of_256": ([3000, 100], 1, 64, 256, 700, 4, 100),
    "everything_stays": ([50, 60], 2, 128, 16, 500, 4, 16),
    "long": ([70001, 20000], 1, 64, 64, 5000, 4, 500),
    "many_requests": ([1 + 7 * i % 190 for i in range(200)], 2, 64, 16, 50, 2, 9),
    "nothing_at_all": ([0, 0], 1, 128, 16, 10, 2, 2),
    "two_ctas_to_a_pair": ([6000, 4097, 5], 2, 64, 64, 1000, 4, 100),
    "four_ctas_to_a_pair": ([12000, 300], 1, 64, 64, 2000, 0, 1),
    "longer_than_the_registers": ([20000] + [3 + i for i in range(76)], 1, 64, 64, 700, 4, 33),
}


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8", "int4"])
@pytest.mark.parametrize("name", list(EVICTS))
def test_the_heaviest_tokens_are_gathered(kind, name):
    from query_aware_sparse_hs_gb300 import hs
    lens, hkv, dim, block, budget, sink, recent = EVICTS[name]
    c = Cache(kind, lens, hkv, dim, block, seed=len(name))
    w = weights_for(c)
    d = destination(c, budget)
    kept = torch.full((len(lens), hkv, budget), 77, dtype=torch.int32, device="cuda")
    hs.hs_evict_tokens(c.shape(2), c.kv, d["kv"], hs.evict_params(budget, sink, recent), w, d["w"], kept)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    check_evicted(c, d, w, budget, sink, recent, kept)
    assert torch.equal(c.gl.cpu(), torch.tensor(lens, dtype=torch.int32))


@pytest.mark.parametrize("n, more", [(900, 0), (7000, 0), (33000, 0), (17000, 80)])  # CTAs to a pair: 1, 2, 8; 1, past its registers
def test_ties_nan_infinities_and_zeros_of_the_weights(n, more):
    from query_aware_sparse_hs_gb300 import hs
    c = Cache("bf16", [n] * 5 + [7] * more, 1, 64, 16, seed=5)
    w = weights_for(c)
    w[0] = 0.5                                  # all alike: the lower ones stay
    w[1, 0, ::2] = -0.0
    w[1, 0, 1::2] = 0.0                         # the same number
    w[2, 0, 100:850] = float("nan")             # last of all
    w[3, 0, 500:700], w[3, 0, 300:400] = float("inf"), float("-inf")
    w[4, 0, :] = -torch.rand(w.shape[2], generator=torch.Generator().manual_seed(1)).cuda()
    for budget, sink, recent in ((300, 4, 64), (64, 0, 0), (n - 1, 1, 1)):
        d = destination(c, budget)
        kept = torch.zeros((5 + more, 1, budget), dtype=torch.int32, device="cuda")
        hs.hs_evict_tokens(c.shape(1), c.kv, d["kv"], hs.evict_params(budget, sink, recent), w, d["w"], kept)
        check_evicted(c, d, w, budget, sink, recent, kept)


def test_lengths_in_place_one_pool_and_no_new_weights():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache("int4", [700, 90, 300], 2, 128, 16, seed=5, spare=120)
    free = np.setdiff1d(np.arange(c.x["k"].shape[0]), c.table[c.table >= 0])
    budget, table = 200, np.full((3, 2, 20), -1, np.int32)
    nb = [13, 6, 13]
    at = 0
    for b in range(3):
        for h in range(2):
            table[b, h, :nb[b]] = free[at:at + nb[b]]
            at += nb[b]
    w = weights_for(c)
    before = {k: (c.x[k].clone(), c.sc[k].clone()) for k in "kv"}
    gt = torch.from_numpy(table).cuda()
    dst = hs.paged_kv(c.x["k"], c.x["v"], gt, c.gl, c.sc["k"], c.sc["v"])
    kept = torch.zeros((3, 2, budget), dtype=torch.int32, device="cuda")
    hs.hs_evict_tokens(c.shape(2), c.kv, dst, hs.evict_params(budget, 4, 32), w, None, kept)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    old = torch.from_numpy(c.table[c.table >= 0].astype(np.int64)).cuda()
    for k in "kv":
        assert torch.equal(c.x[k][old], before[k][0][old]) and torch.equal(c.sc[k][old].view(torch.int16), before[k][1][old].view(torch.int16))
    assert c.gl.tolist() == [200, 90, 200]
    d = {"x": {}, "lens": c.gl, "w": w, "table": table}
    for b, L in enumerate(c.lens):
        for h in range(2):
            t = kept_of(w[b, h].cpu().numpy(), L, budget, 4, 32)
            assert kept[b, h, :len(t)].tolist() == t.tolist()
            i = np.arange(len(t))
            for k in "kv":
                assert torch.equal(c.x[k][torch.from_numpy(c.table[b, h, t // 16].astype(np.int64)).cuda(), torch.from_numpy(t % 16).cuda()],
                                   c.x[k][torch.from_numpy(table[b, h, i // 16].astype(np.int64)).cuda(), torch.from_numpy(i % 16).cuda()])
    del d


def test_pages_out_of_range_and_lengths_past_the_table():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache("bf16", [300, 200], 1, 64, 16, seed=5)
    w = weights_for(c)
    d = destination(c, 64)
    kept = torch.zeros((2, 1, 64), dtype=torch.int32, device="cuda")
    w[0, 0, 160:176] = 50.0  # block 10 stays
    want = kept_of(w[0, 0].cpu().numpy(), 300, 64, 0, 0)
    c.gt[0, 0, 10] = -7
    d["gt"][1, 0, 2] = d["x"]["k"].shape[0]
    hs.hs_evict_tokens(c.shape(1), c.kv, d["kv"], hs.evict_params(64), w, d["w"], kept)
    assert hs.hs_get_device_error()[1] == hs.HS_EBIT_PAGE_RANGE
    assert kept[0, 0].tolist() == want.tolist()
    for i, t in enumerate(want):
        row = d["x"]["k"][d["table"][0, 0, i // 16], i % 16]
        assert torch.equal(row, c.x["k"][c.table[0, 0, t // 16], t % 16]) if t // 16 != 10 else (row == 9).all()
    lost = d["x"]["k"][d["table"][1, 0, 2]]
    assert (lost == 9).all()
    # a request longer than its table: as long as that
    c.gt.copy_(torch.from_numpy(c.table))
    d = destination(c, 64)
    c.gl[1] = 100000
    c.table[1, 0, :] = c.table[1, 0, 0]  # (every block has some page)
    c.gt.copy_(torch.from_numpy(c.table))
    hs.hs_evict_tokens(c.shape(1), c.kv, d["kv"], hs.evict_params(64, 2, 8), w, d["w"], kept)
    assert hs.hs_get_device_error()[1] == hs.HS_EBIT_BLOCK_RANGE
    assert kept[1, 0].tolist() == kept_of(w[1, 0].cpu().numpy(), c.mb * 16, 64, 2, 8).tolist() and d["lens"].tolist() == [64, 64]


def test_captured_and_on_another_stream():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache("int4", [9000, 90], 2, 128, 64, seed=5)
    w = weights_for(c)
    q = queries(c, 8)
    sel, cnt = selection(c, None)
    gsel, gcnt = torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()
    lse = lse_of(c, q, 8, sel, cnt, 128 ** -0.5)
    d = destination(c, 300)
    kept = torch.zeros((2, 2, 300), dtype=torch.int32, device="cuda")

    def both(stream=None):
        hs.hs_accumulate_attn_weights(c.shape(8), c.kv, q, lse, gsel, gcnt, sel.shape[2], 128 ** -0.5, w, stream)
        hs.hs_evict_tokens(c.shape(8), c.kv, d["kv"], hs.evict_params(300, 4, 32), w, d["w"], kept, stream)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    both(side)
    side.synchronize()
    check_evicted(c, d, w, 300, 4, 32, kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (3, 4):
        w.copy_(weights_for(c, seed))
        graph.replay()
        torch.cuda.synchronize()
        check_evicted(c, d, w, 300, 4, 32, kept)


def test_decode_accumulate_evict_and_decode_again():
    """Twelve tokens decoded over a 4-bit cache with the weights accumulated, the cache cut to 160 tokens, and four tokens
    more, at the positions they have in the text: each step's attention against the rows that are there."""
    from query_aware_sparse_hs_gb300 import hs
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    hkv, group, dim, block, budget = 2, 4, 128, 16, 160
    lens = [300, 90]
    c = Cache("int4", lens, hkv, dim, block, seed=6, mb=24, spare=2 * 2 * 24)
    free = list(np.setdiff1d(np.arange(c.x["k"].shape[0]), c.table[c.table >= 0]))
    dec = SparseDecode(num_q_heads=8, num_kv_heads=hkv, head_dim=dim, block_size=block, kv_dtype="int4", batch=2, max_blocks=24,
                       sink_tokens=4, window_tokens=32, k_scored=24, out_is_fp32=True)
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    a = torch.arange(400, dtype=torch.float64)[:, None] * inv
    cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    g = torch.Generator().manual_seed(8)
    weights = torch.zeros((2, hkv, 24 * block), device="cuda")
    text = torch.tensor(lens, dtype=torch.int32).cuda()  # tokens of the text so far

    def pages(cache):
        for b in range(2):
            for h in range(hkv):
                j = (cache.lens[b] - 1) // block
                if cache.table[b, h, j] < 0:
                    cache.table[b, h, j] = free.pop()
        cache.gt.copy_(torch.from_numpy(cache.table))

    def step(cache):
        cache.lens = [n + 1 for n in cache.lens]
        cache.nb = [-(-n // block) for n in cache.lens]
        cache.gl.add_(1)
        pages(cache)
        text.add_(1)
        qkv = torch.randn((2, 8 + 2 * hkv, dim), generator=g).to(torch.bfloat16).cuda()
        q = torch.zeros((2, 8, dim), dtype=torch.bfloat16, device="cuda")
        p = hs.append_params(cos_sin=cos_sin, positions=text - 1)
        dec.append_tokens(cache.kv, p, qkv[:, 8:10], qkv[:, 10:], qkv[:, :8], q)
        dec.select_attend(cache.kv, q)
        start = weights.clone()
        dec.accumulate_weights(cache.kv, q, weights)
        assert hs.hs_get_device_error() == (hs.HS_OK, 0)
        sel, cnt = dec.sel.cpu().numpy(), dec.sel_count.cpu().numpy()
        plain = lse_of(cache, q, group, sel, cnt, dim ** -0.5)
        assert (plain - dec.lse).abs().max() < 1e-4
        for b in range(2):
            for h in range(hkv):
                t = tokens_of(cache, b, sel[b, h, :cnt[b, h]])
                z = q[b, h * group:(h + 1) * group].double().cpu().numpy() @ cache.rows("k", b, h, t).T * dim ** -0.5
                e = np.exp(z - z.max(1, keepdims=True))
                want = e / e.sum(1, keepdims=True) @ cache.rows("v", b, h, t)
                assert np.abs(dec.out[b, h * group:(h + 1) * group].double().cpu().numpy() - want).max() < 1e-4
        check_weights(cache, q, group, dec.lse, sel, cnt, dim ** -0.5, start, weights)

    dec.build_summaries(c.kv)
    for _ in range(12):
        step(c)
    nb = [-(-min(L, budget) // block) for L in c.lens]
    e = Cache.__new__(Cache)
    e.kind, e.hkv, e.d, e.block, e.x, e.sc, e.mb, e.rng = c.kind, hkv, dim, block, c.x, c.sc, 24, c.rng
    e.table = np.full((2, hkv, 24), -1, np.int32)
    for b in range(2):
        for h in range(hkv):
            for j in range(nb[b]):
                e.table[b, h, j] = free.pop()
    e.lens = [min(L, budget) for L in c.lens]
    e.gt, e.gl = torch.from_numpy(e.table).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    e.up()
    after, kept = torch.zeros_like(weights), torch.zeros((2, hkv, budget), dtype=torch.int32, device="cuda")
    dec.evict(c.kv, e.kv, hs.evict_params(budget, 4, 32), weights, after, kept)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0) and e.gl.tolist() == e.lens
    for b in range(2):
        for h in range(hkv):
            t = kept_of(weights[b, h].cpu().numpy(), c.lens[b], budget, 4, 32)
            assert kept[b, h, :len(t)].tolist() == t.tolist()
            assert np.array_equal(e.rows("k", b, h, np.arange(len(t))), c.rows("k", b, h, t))
    weights = after
    for _ in range(4):
        step(e)


# ---- scales that start where an element may ---------------------------------------------------------------------------------


def off_by_words(t, words=1):
    """The same tensor, its first element `words` elements behind a 16-byte boundary."""
    flat = torch.zeros(t.numel() + words, dtype=t.dtype, device=t.device)
    got = flat[words:].view(t.shape)
    got.copy_(t)
    assert got.data_ptr() % 16 == words * t.element_size()
    return got


@pytest.mark.parametrize("words", [1, 2, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_grouped_scales_at_any_element(d, words):
    """Wherever they start, the results are the same."""
    from query_aware_sparse_hs_gb300 import hs
    c = Cache("fp8", [900, 31, 0, 2000], 2, d, 16, seed=4)
    q = queries(c, 8)
    sel, cnt = selection(c, 40, shuffle=True)
    lse = lse_of(c, q, 8, sel, cnt, d ** -0.5)
    start = torch.rand((4, 2, c.mb * 16), generator=torch.Generator().manual_seed(3)).cuda()

    def run():
        got = start.clone()
        hs.hs_accumulate_attn_weights(c.shape(8), c.kv, q, lse, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(),
                                      sel.shape[2], d ** -0.5, got)
        assert hs.hs_get_device_error() == (hs.HS_OK, 0)
        return got

    want = run()
    check_weights(c, q, 8, lse, sel, cnt, d ** -0.5, start, want)
    c.sc["k"] = off_by_words(c.sc["k"], words)
    c.up()
    assert torch.equal(run(), want)


@pytest.mark.parametrize("kind,block", [("bf16", 16), ("int4", 64)])
@pytest.mark.parametrize("on", ["current", "stream", "handle"])
def test_selection_after_an_eviction_with_smoothed_scores(kind, block, on):
    """The first selection over the cut cache is a new decoder's for the requests that were cut, and goes on from its history
    for the one that was not."""
    from query_aware_sparse_hs_gb300 import hs
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    c = Cache(kind, [3000, 250, 2000], 2, 128, block, seed=3)
    e = destination(c, 1024, mb=c.mb)

    def decoder():
        return SparseDecode(num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=block, kv_dtype=kind, batch=3, max_blocks=c.mb,
                            sink_tokens=4, window_tokens=32, k_scored=6, score_smoothing=0.6, out_is_fp32=True)
    dec, fresh, uncut = decoder(), decoder(), decoder()
    for d in (dec, uncut):
        d.build_summaries(c.kv)
        for i in range(3):
            d.step(c.kv, queries(c, 4, seed=20 + i))
    w = weights_for(c)
    kept = torch.zeros((3, 2, 1024), dtype=torch.int32, device="cuda")
    side = None if on == "current" else torch.cuda.Stream()
    stream = side.cuda_stream if on == "handle" else side
    torch.cuda.synchronize()
    dec.evict(c.kv, e["kv"], hs.evict_params(1024, 4, 32), w, None, kept, stream)
    if side is not None:
        torch.cuda.current_stream().wait_stream(side)
    fresh.build_summaries(e["kv"])
    q = queries(c, 4, seed=40)
    dec.step(e["kv"], q)
    fresh.step(e["kv"], q)
    uncut.step(c.kv, q)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    for b, other in ((0, fresh), (1, uncut), (2, fresh)):
        n = -(-min(c.lens[b], 1024) // block)
        assert torch.equal(dec.sel[b], other.sel[b]), b
        assert other is uncut or torch.equal(dec.out[b], other.out[b]), b  # (over the old cache the work may be cut elsewhere)
        assert torch.equal(dec.score_history[b, :, :n], other.score_history[b, :, :n]), b
    assert dec.score_history[[0, 2], :, -(-1024 // block):].isnan().all()


def test_weights_that_take_turns_between_two_buffers():
    """Accumulate, cut, accumulate, cut back into the first buffer, whose old weights lie behind the new lengths: tokens that
    come then start at 0."""
    from query_aware_sparse_hs_gb300 import hs
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    c = Cache("bf16", [900, 150, 40], 2, 64, 16, seed=3)
    dec = SparseDecode(num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16, kv_dtype="bf16", batch=3, max_blocks=c.mb,
                       sink_tokens=4, window_tokens=32, k_scored=90)
    bufs = [torch.zeros((3, 2, c.mb * 16), device="cuda"), torch.full((3, 2, c.mb * 16), 5.0, device="cuda")]
    now = c
    for i, budget in enumerate((200, 100)):
        dec.build_summaries(now.kv)
        q = queries(now, 4, seed=i)
        dec.step(now.kv, q)
        dec.accumulate_weights(now.kv, q, bufs[0])
        d = destination(now, budget, mb=c.mb)
        kept = torch.zeros((3, 2, budget), dtype=torch.int32, device="cuda")
        dec.evict(now.kv, d["kv"], hs.evict_params(budget, 4, 32), bufs[0], bufs[1], kept)
        assert hs.hs_get_device_error() == (hs.HS_OK, 0)
        lens = [min(n, budget) for n in now.lens]
        for b, n in enumerate(lens):
            for h in range(2):
                t = kept_of(bufs[0][b, h].cpu().numpy(), now.lens[b], budget, 4, 32)
                assert torch.equal(bufs[1][b, h, :n], bufs[0][b, h, torch.from_numpy(t).cuda()])
                assert (bufs[1][b, h, n:] == 0).all(), (i, b, h)
        nxt = Cache.__new__(Cache)
        nxt.kind, nxt.hkv, nxt.d, nxt.block, nxt.mb, nxt.rng = "bf16", 2, 64, 16, c.mb, c.rng
        nxt.x, nxt.sc, nxt.table, nxt.gt, nxt.gl, nxt.lens = d["x"], d["sc"], d["table"], d["gt"], d["lens"], lens
        nxt.up()
        now = nxt
        bufs.reverse()


def nobody_is_written(c, d, budget):
    """Scales of rows that no request has still hold their fill (the rows themselves: check_evicted)."""
    for k in "kv":
        free = torch.ones(d["x"][k].shape[:2], dtype=torch.bool)
        for b, L in enumerate(c.lens):
            i = np.arange(min(L, budget))
            for h in range(c.hkv):
                free[d["table"][b, h, i // c.block], i % c.block] = False
        assert free.any() and (d["sc"][k].float()[free.cuda()] == 9).all()


@pytest.mark.parametrize("src,dst", [(0, 0), (1, 0), (0, 1), (2, 2), (3, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_grouped_scales_at_any_element_are_gathered(d, src, dst):
    """Scales that start `src` and `dst` elements behind a boundary: by 16 or 8 bytes where all of them allow it, else by 4."""
    from query_aware_sparse_hs_gb300 import hs
    c = Cache("fp8", [900, 100, 3], 2, d, 16, seed=5)
    w = weights_for(c)
    e = destination(c, 130)
    for k, other in (("k", 0), ("v", 1)):
        c.sc[k] = off_by_words(c.sc[k], src)
        e["sc"][k] = off_by_words(e["sc"][k], (dst + other) % 4 if dst == 1 else dst)
    c.up()
    e["kv"] = hs.paged_kv(e["x"]["k"], e["x"]["v"], e["gt"], e["lens"], e["sc"]["k"], e["sc"]["v"])
    kept = torch.full((3, 2, 130), 77, dtype=torch.int32, device="cuda")
    hs.hs_evict_tokens(c.shape(2), c.kv, e["kv"], hs.evict_params(130, 4, 32), w, e["w"], kept)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    check_evicted(c, e, w, 130, 4, 32, kept)
    nobody_is_written(c, e, 130)


@pytest.mark.parametrize("kind", ["int4", "fp8"])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 16), (128, 5)])
def test_scales_and_centres_are_gathered_within_one_pool(kind, d, block):
    """Source and destination pages of one pool: codes, scales and centres arrive bit for bit, everything else stays."""
    from query_aware_sparse_hs_gb300 import hs
    budget = 200
    nb = [-(-min(L, budget) // block) for L in (700, 90, 300)]
    c = Cache(kind, [700, 90, 300], 2, d, block, seed=5, spare=2 * sum(nb) + 7)
    free = list(np.setdiff1d(np.arange(c.x["k"].shape[0]), c.table[c.table >= 0]))
    table = np.full((3, 2, max(nb)), -1, np.int32)
    for b in range(3):
        for h in range(2):
            table[b, h, :nb[b]] = [free.pop() for _ in range(nb[b])]
    w = weights_for(c)
    want = {k: (c.x[k].clone().view(torch.uint8), c.sc[k].clone().view(torch.uint8)) for k in "kv"}
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    dst = hs.paged_kv(c.x["k"], c.x["v"], torch.from_numpy(table).cuda(), lens, c.sc["k"], c.sc["v"])
    kept = torch.zeros((3, 2, budget), dtype=torch.int32, device="cuda")
    hs.hs_evict_tokens(c.shape(2), c.kv, dst, hs.evict_params(budget, 4, 32), w, None, kept)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0) and lens.tolist() == [200, 90, 200]
    for b, L in enumerate(c.lens):
        for h in range(2):
            t = kept_of(w[b, h].cpu().numpy(), L, budget, 4, 32)
            i = np.arange(len(t))
            src = torch.from_numpy(c.table[b, h, t // block].astype(np.int64)).cuda(), torch.from_numpy(t % block).cuda()
            to = torch.from_numpy(table[b, h, i // block].astype(np.int64)).cuda(), torch.from_numpy(i % block).cuda()
            for k in "kv":
                for x in want[k]:
                    x[to] = x[src]
    for k in "kv":
        assert torch.equal(c.x[k].view(torch.uint8), want[k][0]) and torch.equal(c.sc[k].view(torch.uint8), want[k][1])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_weights_and_eviction_of_pools_past_four_gib(kind):
    """Rows, and for eviction the rows they go to, beyond 2^32 bytes of their pool: the same as from a small one."""
    from query_aware_sparse_hs_gb300 import hs
    c = Cache(kind, [700, 130], 2, 128, 64, seed=5)
    q = queries(c, 8)
    sel, cnt = selection(c, None)
    lse = lse_of(c, q, 8, sel, cnt, 128 ** -0.5)
    d = destination(c, 300)
    w = weights_for(c)
    total = (1 << 32) // (64 * 128 * c.x["k"].element_size()) + 200
    far = np.random.default_rng(1).permutation(np.arange(total - 190, total))
    pages, more = c.x["k"].shape[0], d["x"]["k"].shape[0]

    def pool(x, at):
        if x is None:
            return None
        big = torch.full((total,) + x.shape[1:], 9, dtype=x.dtype, device="cuda")
        big[torch.from_numpy(at).cuda()] = x
        return big

    def moved(table, at):
        return torch.from_numpy(np.where(table >= 0, at[np.maximum(table, 0)], -1).astype(np.int32)).cuda()

    x, sc = {k: pool(c.x[k], far[:pages]) for k in "kv"}, {k: pool(c.sc[k], far[:pages]) for k in "kv"}
    src = hs.paged_kv(x["k"], x["v"], moved(c.table, far[:pages]), c.gl, sc["k"], sc["v"])
    at = far[pages:pages + more]
    to = hs.paged_kv(x["k"], x["v"], moved(d["table"], at), d["lens"], sc["k"], sc["v"])
    got = [torch.zeros((2, 2, c.mb * 64), device="cuda") for _ in range(2)]
    for kv, g in zip((c.kv, src), got):
        hs.hs_accumulate_attn_weights(c.shape(8), kv, q, lse, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(), sel.shape[2],
                                      128 ** -0.5, g)
    check_weights(c, q, 8, lse, sel, cnt, 128 ** -0.5, torch.zeros_like(got[0]), got[0])
    assert torch.equal(got[0], got[1])
    kept = torch.zeros((2, 2, 300), dtype=torch.int32, device="cuda")
    hs.hs_evict_tokens(c.shape(8), src, to, hs.evict_params(300, 4, 32), w, d["w"], kept)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    for k in "kv":
        d["x"][k] = x[k][torch.from_numpy(at).cuda()]
        if sc[k] is not None:
            d["sc"][k] = sc[k][torch.from_numpy(at).cuda()]
    check_evicted(c, d, w, 300, 4, 32, kept)


def test_the_driver_captured_and_on_the_default_stream_by_its_handle():
    """A captured evict() clears the weights and the smoothed scores at every replay; handle 0 is the default stream."""
    from query_aware_sparse_hs_gb300 import hs
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    c = Cache("int4", [900, 150], 2, 64, 16, seed=3)
    dec = SparseDecode(num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16, kv_dtype="int4", batch=2, max_blocks=c.mb,
                       sink_tokens=4, window_tokens=32, k_scored=9, score_smoothing=0.5)
    d = destination(c, 200, mb=c.mb)
    kept = torch.zeros((2, 2, 200), dtype=torch.int32, device="cuda")
    w = weights_for(c)

    def evict(stream=None):
        dec.evict(c.kv, d["kv"], hs.evict_params(200, 4, 32), w, d["w"], kept, stream)

    def before(seed):
        w.copy_(weights_for(c, seed))
        d["w"].fill_(7.0)
        dec.score_history.copy_(torch.rand(dec.score_history.shape))
        return dec.score_history.clone()

    def after(old):
        torch.cuda.synchronize()
        assert hs.hs_get_device_error() == (hs.HS_OK, 0)
        assert dec.score_history[0].isnan().all() and torch.equal(dec.score_history[1], old[1])
        for b, n in enumerate((200, 150)):
            assert (d["w"][b, :, n:] == 0).all()
            for h in range(2):
                t = kept_of(w[b, h].cpu().numpy(), c.lens[b], 200, 4, 32)
                assert torch.equal(d["w"][b, h, :n], w[b, h, torch.from_numpy(t).cuda()])

    old = before(1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        evict(0)
    after(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        evict()
    for seed in (2, 3):
        old = before(seed)
        graph.replay()
        after(old)
