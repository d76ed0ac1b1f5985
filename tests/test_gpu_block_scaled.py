"""The e4m3 cache with one scale per page: attention over it (tensor-core and CUDA-core), its block summaries, and whole
decode steps on it, against plain 64-bit loops.  GPU only."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -23  # a rounding of an fp32 sum on the matrix units (truncation counted)


class Cache:
    def __init__(self, lens, hkv, d, block, seed=0, kscale=(-9, -5), vscale=(-9, -5), poison=True, spare=2):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.hkv, self.d, self.block = rng, list(lens), hkv, d, block
        self.nb = [-(-n // block) for n in lens]
        self.mb = max(1, max(self.nb)) + 1
        self.pages = sum(self.nb) * hkv + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), hkv, self.mb), -1, np.int32)
        at = 0
        for b, n in enumerate(self.nb):
            for h in range(hkv):
                self.table[b, h, :n] = order[at:at + n]
                at += n
        shape = (self.pages, block, d)
        self.codes = {w: O.e4m3_encode(rng.standard_normal(shape) * 90) for w in "kv"}
        self.scales = {w: np.exp2(rng.uniform(*e, self.pages)).astype(np.float32) for w, e in (("k", kscale), ("v", vscale))}
        if poison:  # rows behind the last token, and pages of nobody, hold NaN
            for b, L in enumerate(lens):
                if L % block:
                    for h in range(hkv):
                        for w in "kv":
                            self.codes[w][self.table[b, h, L // block], L % block:] = 0x7F
            for p in order[at:]:
                for w in "kv":
                    self.codes[w][p] = 0xFF
                    self.scales[w][p] = np.nan
        self.up()

    def up(self):
        from query_aware_sparse_hs_gb300 import hs
        c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.g = {w: c(self.codes[w]) for w in "kv"}
        self.gs = {w: c(self.scales[w]) for w in "kv"}
        self.gt, self.gl = c(self.table), torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.kv = hs.paged_kv(self.g["k"], self.g["v"], self.gt, self.gl, self.gs["k"], self.gs["v"])

    def rows(self, w, b, h, blocks):
        """64-bit values of the valid tokens of `blocks`."""
        out = [np.zeros((0, self.d))]
        for j in blocks:
            n = min(self.block, self.lens[b] - j * self.block)
            p = self.table[b, h, j]
            out.append(O.e4m3_decode(self.codes[w][p, :n]) * float(self.scales[w][p]))
        return np.concatenate(out)


def chosen(c, capacity, keep, shuffle=False):
    """sel and sel_count: `keep` blocks of each (request, kv head) (None: all)."""
    sel = np.full((len(c.lens), c.hkv, capacity), -1, np.int32)
    cnt = np.zeros((len(c.lens), c.hkv), np.int32)
    for b, n in enumerate(c.nb):
        for h in range(c.hkv):
            k = n if keep is None else min(n, keep if isinstance(keep, int) else keep[b])
            got = c.rng.permutation(n)[:k]
            sel[b, h, :k] = got if shuffle else np.sort(got)
            cnt[b, h] = k
    return sel, cnt


def attend(c, q, sel, cnt, f32=True, counters=True, algo="auto", max_ctas=0, scale=None, bps=0, lse=True):
    from query_aware_sparse_hs_gb300 import hs
    hq = q.shape[1]
    shape = hs.attn_shape(hq, c.hkv, c.d, c.block, "fp8_block")
    ctr = torch.zeros(len(c.lens) * c.hkv, dtype=torch.int32, device="cuda") if counters else None
    p = hs.attn_params(c.d ** -0.5 if scale is None else scale, f32, bps, algo, max_ctas, split_counters=ctr)
    ws = torch.full((max(256, hs.hs_workspace_bytes(shape, len(c.lens), sel.shape[2], p)),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, 3.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:2], 3.0, device="cuda") if lse else None
    hs.hs_sparse_paged_decode_attn(shape, c.kv, q, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(), sel.shape[2], p,
                                   out, ls, ws)
    if ctr is not None:
        assert (ctr == 0).all()
    return out, ls


def check_attention(c, q, sel, cnt, out, lse, scale=None, simt=False):
    """Against the definition.  Bounds: a logit is a sum of D fp32-rounded terms (D U of the sum of magnitudes, and the
    query's entries exact to 2^-33 of the largest), times two factors; P's two f16 terms hold 2^-21 of it, or 2^-39 of
    the largest V scale met (one term, 2^-11 or 2^-39, for bf16 outputs); an output is a sum of T such terms."""
    scale = c.d ** -0.5 if scale is None else scale
    qn, group = q.double().cpu().numpy(), q.shape[1] // c.hkv
    half = 0.0 if out.dtype == torch.float32 else 2.0 ** -8
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(c.lens)):
        for h in range(c.hkv):
            blocks = sel[b, h, :cnt[b, h]]
            K, V = c.rows("k", b, h, blocks), c.rows("v", b, h, blocks)
            T = len(K)
            for i in range(h * group, (h + 1) * group):
                if T == 0:
                    assert (got[b, i] == 0).all() and gl[b, i] == -np.inf
                    continue
                s = K @ qn[b, i] * scale
                mags = (np.abs(K) @ np.abs(qn[b, i]) + np.abs(K).sum(1) * np.abs(qn[b, i]).max() * 2.0 ** -33) * abs(scale)
                ds = (mags * (c.d * U + 4 * U)).max() + 4 * U * np.abs(s).max()
                m = s.max()
                p = np.exp(s - m)
                want, l = (p[:, None] * V).sum(0) / p.sum(), m + math.log(p.sum())
                assert abs(gl[b, i] - l) <= ds + (T + 40) * U + 4 * U * abs(l), (b, i, gl[b, i], l)
                weight = (p[:, None] * np.abs(V)).sum(0) / p.sum()
                rel = 2 * math.expm1(ds) + (T + 60) * U + (2.0 ** -20 if half == 0 or simt else 2.0 ** -11)
                tiny = 0.0 if simt else 448 * 2.0 ** -38 * float(np.max([c.scales["v"][c.table[b, h, j]] for j in blocks]))
                bound = half * np.abs(want) + (1 + half) * (rel * weight + tiny * T / p.sum())
                assert (np.abs(got[b, i] - want) <= bound).all(), (b, i, np.abs(got[b, i] - want).max(), bound.min())


def query(c, hq, seed=1, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((len(c.lens), hq, c.d), generator=g) * torch.exp2(spread * torch.randn((len(c.lens), hq, 1), generator=g))
    return q.to(torch.bfloat16).cuda()


CASES = {
    # request lengths, kv heads, group, d, block, blocks kept (None: all), order
    "one_token": ([1], 1, 8, 128, 64, None, False),
    "around_a_tile": ([31, 32, 33, 63, 64, 65], 2, 8, 128, 64, None, False),
    "pages_of_16": ([1, 17, 500, 1000], 2, 4, 128, 16, None, False),
    "pages_of_16_selected": ([900, 30, 2000], 1, 8, 128, 16, 7, False),
    "any_order": ([900, 30, 2000], 2, 8, 128, 32, 9, True),
    "pages_of_one": ([5, 40], 1, 2, 128, 1, None, False),
    "pages_of_five": ([3, 44, 201], 2, 1, 128, 5, None, False),
    "pages_of_48": ([48, 47, 700], 1, 16, 128, 48, None, False),
    "pages_of_256": ([255, 257, 1024], 1, 8, 128, 256, None, False),
    "group_16": ([700, 3, 65], 2, 16, 128, 64, None, False),
    "d64": ([700, 3, 65], 2, 8, 64, 64, None, False),
    "d64_group_16": ([333, 1, 64], 1, 16, 64, 16, None, False),
    "d64_group_1_pages_of_7": ([333, 6, 64], 3, 1, 64, 7, None, True),
    "empty_requests": ([0, 100, 0, 0, 5, 0], 2, 8, 128, 16, None, False),
    "nothing_selected": ([100, 200], 2, 8, 128, 16, 0, False),
    "one_long_among_short": ([20000] + [3] * 20, 1, 8, 128, 64, None, False),
    "many_requests": ([1 + 7 * i % 90 for i in range(400)], 2, 2, 64, 16, None, False),
    "one_kv_head_long": ([30011], 1, 8, 128, 32, None, False),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("form", ["merge_in_place", "merge_launch", "bf16_out", "simt"])
def test_attention_matches_the_definition(name, form):
    lens, hkv, group, d, block, keep, shuffle = CASES[name]
    c = Cache(lens, hkv, d, block, seed=len(name))
    q = query(c, hkv * group, spread=1.0)
    sel, cnt = chosen(c, max(1, max(c.nb)) if keep is None else max(1, keep), keep, shuffle)
    simt = form == "simt"
    out, lse = attend(c, q, sel, cnt, f32=form != "bf16_out", counters=form != "merge_launch", algo="simt" if simt else "auto")
    from query_aware_sparse_hs_gb300 import hs
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    check_attention(c, q, sel, cnt, out, lse, simt=simt)


@pytest.mark.parametrize("group,d", [(8, 128), (16, 128), (2, 64), (16, 64)])
def test_bf16_outputs_are_the_fp32_outputs_rounded(group, d):
    """The output's type decides its last rounding and nothing before it."""
    c = Cache([3000, 100, 700], 2, d, 64, seed=12)
    q = query(c, 2 * group)
    sel, cnt = chosen(c, max(c.nb), None)
    for counters in (True, False):
        wide, lw = attend(c, q, sel, cnt, counters=counters)
        out, lse = attend(c, q, sel, cnt, f32=False, counters=counters)
        assert torch.equal(out, wide.to(torch.bfloat16)) and torch.equal(lse, lw)


def test_results_do_not_depend_on_the_arrival_order_or_the_number_of_ctas():
    c = Cache([9000, 100, 5000], 2, 128, 64, seed=3)
    q = query(c, 16)
    sel, cnt = chosen(c, max(c.nb), None)
    a, la = attend(c, q, sel, cnt)
    for _ in range(20):
        b, lb = attend(c, q, sel, cnt)
        assert torch.equal(a, b) and torch.equal(la, lb)
    m, lm = attend(c, q, sel, cnt, counters=False)
    assert torch.equal(a, m) and torch.equal(la, lm)
    for n in (1, 2, 7):
        b, lb = attend(c, q, sel, cnt, max_ctas=n)
        check_attention(c, q, sel, cnt, b, lb)
    b, _ = attend(c, q, sel, cnt, lse=False, bps=5)
    assert torch.equal(a, b)
    # hundreds of pairs to a CTA, a long one among them
    c = Cache([1 + 7 * i % 90 for i in range(150)] + [3000], 2, 64, 16, seed=3)
    q = query(c, 4)
    sel, cnt = chosen(c, max(c.nb), None)
    for n in (1, 3, 0):
        for counters in (True, False):
            b, lb = attend(c, q, sel, cnt, max_ctas=n, counters=counters)
            check_attention(c, q, sel, cnt, b, lb)


@pytest.mark.parametrize("vscale", [(-30, 4), (-60, -55), (10, 14)])
def test_v_scales_of_very_different_sizes(vscale):
    c = Cache([700, 64, 2000], 1, 128, 16, seed=4, vscale=vscale)
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt)
    check_attention(c, q, sel, cnt, out, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_a_v_scale_near_the_largest_float(d):
    c = Cache([100, 64], 1, d, 64, seed=4, poison=False)
    c.scales["v"][c.table[0, 0, 0]] = 1.75 * 2.0 ** 127
    c.codes["v"][c.table[0, 0, 0]] = O.e4m3_encode(c.rng.uniform(-1, 1, (64, d)))
    c.up()
    q = query(c, 8)
    sel, cnt = chosen(c, 2, None)
    out, lse = attend(c, q, sel, cnt)
    assert torch.isfinite(out).all()
    check_attention(c, q, sel, cnt, out, lse)


def test_v_scales_near_the_smallest():
    c = Cache([700, 64, 2000], 1, 128, 16, seed=4, vscale=(-111, -108))
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt)
    check_attention(c, q, sel, cnt, out, lse)


@pytest.mark.parametrize("d,group", [(128, 8), (64, 16)])
@pytest.mark.parametrize("top", [1.0, 1.9921875, 2.0 ** 100, 2.0 ** -100, 2.0 ** -117])
def test_small_entries_of_a_query_are_held_to_2_33_of_the_largest(d, group, top):
    """One token, so that lse is its logit: the query's largest entry meets a zero of K, a small one the largest code."""
    c = Cache([1], 1, d, 16, seed=1, poison=False)
    c.codes["k"][c.table[0, 0, 0], 0] = 0
    c.codes["k"][c.table[0, 0, 0], 0, 1] = 0x7E  # 448
    c.scales["k"][:] = 2.0 ** 24
    c.up()
    sel, cnt = chosen(c, 1, None)
    q = torch.zeros((1, group, d), dtype=torch.float64)
    q[:, :, 0] = top
    for h in range(group):
        q[:, h, 1] = top * 2.0 ** -(24 + h) * 1.5
    q = q.to(torch.bfloat16).cuda()
    out, lse = attend(c, q, sel, cnt, scale=1.0 / top)
    qn = q.double().cpu().numpy()[0]
    want = qn[:, 1] * 448 * 2.0 ** 24 / top
    # half a step of f16's smallest numbers; the products are exact, then four roundings of fp32
    err = np.where(qn[:, 1] >= 2.0 ** -25 * top, 0.0, 2.0 ** -33 * 448 * 2.0 ** 24) + 8 * U * np.abs(want)
    assert (np.abs(lse[0].double().cpu().numpy() - want) <= err).all()


def test_queries_at_the_end_of_bf16_are_exact():
    c = Cache([1], 1, 64, 16, seed=1, poison=False)
    c.codes["k"][c.table[0, 0, 0], 0] = 0
    c.codes["k"][c.table[0, 0, 0], 0, 1] = 0x7E
    c.scales["k"][:] = 2.0 ** 90
    c.up()
    sel, cnt = chosen(c, 1, None)
    for top in (2.0 ** -119, 1.9921875 * 2.0 ** -119, 2.0 ** -126, 2.0 ** -133):
        q = torch.zeros((1, 8, 64), dtype=torch.float64)
        q[:, :, 0], q[:, :, 1] = top, 2.0 ** -133
        q = q.to(torch.bfloat16).cuda()
        out, lse = attend(c, q, sel, cnt, scale=2.0 ** 36)
        want = float(q[0, 0, 1].double()) * 448 * 2.0 ** 126
        assert want == 3.5 and (lse - want).abs().max() <= 8 * U * want


@pytest.mark.parametrize("q0,kscale", [(2.0 ** -118, 2.0 ** 100), (2.0 ** -126, 2.0 ** 100), (2.0 ** -100, 2.0 ** 90), (2.0 ** 110, 2.0 ** -117)])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 12, -1.0, 0.0])
def test_logits_of_tiny_queries_and_large_k_scales(q0, kscale, scale):
    """The factor of the logits is very small where the query is, whatever the K scale makes of it."""
    c = Cache([2], 1, 64, 16, seed=1, poison=False)
    page = c.table[0, 0, 0]
    c.codes["k"][page, :2] = 0
    c.codes["k"][page, 0, 0], c.codes["k"][page, 1, 0] = 0x7E, 0xFE  # 448, -448
    c.scales["k"][:] = kscale
    c.up()
    sel, cnt = chosen(c, 1, None)
    q = torch.zeros((1, 8, 64), dtype=torch.float64)
    q[:, :, 0] = q0
    q = q.to(torch.bfloat16).cuda()
    out, lse = attend(c, q, sel, cnt, scale=scale)
    logit = q0 * 448 * kscale * abs(scale)
    want = logit + math.log1p(math.exp(-2 * logit))
    # the factor may lie under fp32's normal numbers: half of 2^-149 times the largest product of codes and scale
    tiny = 2.0 ** -149 * 448 * 512 * kscale
    assert (lse - want).abs().max() <= 8 * U * (abs(want) + 1) + 2 * tiny, (lse[0, 0], want)


@pytest.mark.parametrize("kscale,f", [((99, 100), -104), ((-117, -116), 110)])
def test_k_scales_at_the_ends_of_their_range(kscale, f):
    c = Cache([700, 64, 33], 1, 128, 16, seed=4, kscale=kscale)
    q = query(c, 8) * 2.0 ** f
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt, scale=2.0 ** -4)
    check_attention(c, q, sel, cnt, out, lse, scale=2.0 ** -4)


def test_pages_of_zeros_and_large_or_tiny_queries():
    c = Cache([300, 64], 1, 128, 16, seed=4, poison=False)
    for p in c.table[0, 0, 3:9]:  # as the append leaves a page of zeros
        c.codes["v"][p] = 0
        c.scales["v"][p] = 2.0 ** -117
    c.codes["k"][c.table[1, 0, :4]] = 0
    c.scales["k"][c.table[1, 0, :4]] = 2.0 ** -117
    c.up()
    sel, cnt = chosen(c, max(c.nb), None)
    for f in (1.0, 2.0 ** 60, 2.0 ** -60, 2.0 ** -126, 0.0):
        q = query(c, 8) * f
        # logits of ordinary size whatever the query's
        scale = 0.0 if f == 0 else 128 ** -0.5 / f if f > 2.0 ** -100 else 128 ** -0.5
        out, lse = attend(c, q, sel, cnt, scale=scale)
        check_attention(c, q, sel, cnt, out, lse, scale=scale)


def test_large_logits_of_either_sign():
    c = Cache([500], 1, 128, 64, seed=5, kscale=(-2, 0))
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    for scale in (1.0, -1.0):
        out, lse = attend(c, q, sel, cnt, scale=scale)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        check_attention(c, q, sel, cnt, out, lse, scale=scale)


def test_not_a_number_in_a_selected_row_reaches_only_its_own_outputs():
    c = Cache([100, 100], 2, 128, 16, seed=6)
    c.codes["v"][c.table[0, 1, 2], 5, 7] = 0x7F
    c.up()
    q = query(c, 4)
    sel, cnt = chosen(c, max(c.nb), None)
    for algo in ("auto", "simt"):
        out, lse = attend(c, q, sel, cnt, algo=algo)
        bad = torch.isnan(out)
        assert bad[0, 2:, 7].all() and bad.sum() == 2 and torch.isfinite(lse).all()
    c.codes["k"][c.table[0, 1, 2], 5, 7] = 0xFF
    c.up()
    out, lse = attend(c, q, sel, cnt)
    assert torch.isnan(out[0, 2:]).all() and torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()


def test_requests_of_nothing_but_not_a_number():
    for lens in ([1, 40], [9000, 40]):  # one CTA, and several merged
        c = Cache(lens, 1, 128, 16, seed=6)
        n = -(-lens[0] // 16)
        c.codes["k"][c.table[0, 0, :n]] = 0x7F
        c.up()
        q = query(c, 4)
        sel, cnt = chosen(c, max(c.nb), None)
        for counters in (True, False):
            out, lse = attend(c, q, sel, cnt, counters=counters)
            assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and torch.isfinite(out[1]).all()


def test_bad_selections_and_pages_are_reported_and_skipped():
    from query_aware_sparse_hs_gb300 import hs
    for algo in ("auto", "simt"):
        c = Cache([100, 100], 1, 128, 16, seed=7)
        q = query(c, 8)
        sel, cnt = chosen(c, max(c.nb), None)
        good, lse = attend(c, q, sel, cnt, algo=algo)
        bad = sel.copy()
        bad[0, 0, 3] = c.nb[0]  # past the request
        bad[0, 0, 4] = -7
        out, _ = attend(c, q, bad, cnt, algo=algo)
        assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, hs.HS_EBIT_BLOCK_RANGE)
        assert torch.equal(out[1], good[1])
        left = np.delete(sel[0, 0], [3, 4])
        part, pl = sel.copy(), cnt.copy()
        part[0, 0, :len(left)] = left
        pl[0, 0] = len(left)
        check_attention(c, q, part, pl, out, attend(c, q, part, pl, algo=algo)[1])
        c.gt[0, 0, 3], c.gt[0, 0, 4] = -1, c.pages
        out2, _ = attend(c, q, sel, cnt, algo=algo)
        assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, hs.HS_EBIT_PAGE_RANGE)
        assert torch.equal(out2[1], good[1])
        big = cnt.copy()
        big[1, 0] = sel.shape[2] + 9  # counted past the capacity: cut off there
        out3, _ = attend(c, q, sel, big, algo=algo)
        bits = hs.hs_get_device_error()[1]
        assert bits & hs.HS_EBIT_CAPACITY
        assert torch.equal(out3[1], good[1])


@pytest.mark.parametrize("entry", [-2 ** 31, -2 ** 31 + 1, -1, 2 ** 31 - 1])
def test_every_entry_outside_the_request_is_reported(entry):
    from query_aware_sparse_hs_gb300 import hs
    for algo in ("auto", "simt"):
        c = Cache([1000, 100], 1, 128, 16, seed=7)
        q = query(c, 8)
        sel, cnt = chosen(c, max(c.nb), None)
        bad = sel.copy()
        bad[0, 0, 40] = entry
        out, lse = attend(c, q, bad, cnt, algo=algo)
        assert hs.hs_get_device_error() == (hs.HS_ERR_OUT_OF_RANGE, hs.HS_EBIT_BLOCK_RANGE)
        part, less = sel.copy(), cnt.copy()
        part[0, 0, :62] = np.delete(sel[0, 0], 40)
        less[0, 0] = 62
        check_attention(c, q, part, less, out, lse, simt=algo == "simt")


def test_a_block_selected_twice_counts_twice():
    c = Cache([500], 1, 128, 16, seed=7)
    q = query(c, 8)
    sel = np.array([[[3, 3, 31, 0, 31, 31]]], np.int32)
    cnt = np.array([[6]], np.int32)
    for algo in ("auto", "simt"):
        out, lse = attend(c, q, sel, cnt, algo=algo)
        check_attention(c, q, sel, cnt, out, lse, simt=algo == "simt")


def test_no_allocation_call_and_workspace_checks():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache([300, 200], 2, 128, 64, seed=8)
    q = query(c, 16)
    sel, cnt = chosen(c, max(c.nb), None)
    want, wl = attend(c, q, sel, cnt)
    shape = hs.attn_shape(16, 2, 128, 64, "fp8_block")
    p = hs.attn_params(128 ** -0.5, True)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    gs, gc = torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()
    hs.hs_sparse_paged_decode_attn_noalloc(shape, c.kv, q, gs, gc, sel.shape[2], p, out, lse)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    need = hs.hs_workspace_bytes(shape, 2, sel.shape[2], p)
    for ws in (None, torch.empty(need // 8, dtype=torch.uint8, device="cuda")):
        with pytest.raises(hs.HSError) as e:
            hs.hs_sparse_paged_decode_attn(shape, c.kv, q, gs, gc, sel.shape[2], p, out, lse, ws)
        assert e.value.status == hs.HS_ERR_WORKSPACE


def test_captured_and_replayed_with_other_lengths_and_on_another_stream():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache([900, 70], 2, 128, 16, seed=9)
    q = query(c, 16)
    sel, cnt = chosen(c, max(c.nb), None)
    shape = hs.attn_shape(16, 2, 128, 16, "fp8_block")
    ctr = torch.zeros(4, dtype=torch.int32, device="cuda")
    p = hs.attn_params(128 ** -0.5, True, split_counters=ctr)
    ws = torch.empty(hs.hs_workspace_bytes(shape, 2, sel.shape[2], p), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    gs, gc = torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_sparse_paged_decode_attn(shape, c.kv, q, gs, gc, sel.shape[2], p, out, lse, ws)
    for lens in ([900, 70], [890, 1], [1, 65]):
        c.lens = lens
        c.gl.copy_(torch.tensor(lens, dtype=torch.int32))
        for b in range(2):
            n = -(-lens[b] // 16)
            cnt[b] = n
            sel[b, :, :n] = np.arange(n)
        gs.copy_(torch.from_numpy(sel))
        gc.copy_(torch.from_numpy(cnt))
        for b in range(2):  # rows behind the shorter request are others' from now on
            pass
        graph.replay()
        check_attention(c, q, sel, cnt, out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = torch.empty_like(out)
    with torch.cuda.stream(side):
        hs.hs_sparse_paged_decode_attn(shape, c.kv, q, gs, gc, sel.shape[2], p, again, lse, ws)
    side.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("long", [1, 3000])
def test_thousands_of_requests(long):
    """More pairs than threads of a CTA, hundreds of them empty, one long or none."""
    lens = [(3 * i) % 41 for i in range(2500)]
    lens[1777] = long
    c = Cache(lens, 1, 64, 16, seed=13)
    q = query(c, 2)
    sel, cnt = chosen(c, max(c.nb), None)
    for counters in (True, False):
        out, lse = attend(c, q, sel, cnt, counters=counters)
        check_attention(c, q, sel, cnt, out, lse)
    from query_aware_sparse_hs_gb300 import hs
    lo = torch.full((2500, 1, c.mb, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    hi = lo.clone()
    hs.hs_build_block_summaries(hs.attn_shape(2, 1, 64, 16, "fp8_block"), c.kv, 0, lo, hi)
    lo, hi = lo.double().cpu().numpy(), hi.double().cpu().numpy()
    for b, n in enumerate(c.nb):
        assert (lo[b, 0, n:] == 9).all() and (hi[b, 0, n:] == 9).all()
        for j in range(n):
            x = c.rows("k", b, 0, [j]).astype(np.float32)
            assert np.array_equal(lo[b, 0, j], O.bf16_round_down(x.min(0))) and np.array_equal(hi[b, 0, j], O.bf16_round_up(x.max(0)))


def test_two_calls_at_once_with_their_own_workspaces():
    a, b = Cache([5000, 70], 2, 128, 16, seed=9), Cache([20, 9000, 3], 1, 64, 64, seed=10)
    qa, qb = query(a, 16), query(b, 16)
    want = [attend(a, qa, *chosen(a, max(a.nb), None)), attend(b, qb, *chosen(b, max(b.nb), None))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, c, q in zip(streams, (a, b), (qa, qb)):
            with torch.cuda.stream(s):
                got.append(attend(c, q, *chosen(c, max(c.nb), None)))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


SECOND_CONTEXT = """
import ctypes, math
import numpy as np
from query_aware_sparse_hs_gb300 import hs
cu = ctypes.CDLL("libcuda.so.1")

def ok(status):
    assert status == 0, status

def on_gpu(a):
    p = ctypes.c_uint64()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(a.nbytes)))
    ok(cu.cuMemcpyHtoD_v2(p, a.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(a.nbytes)))
    return p.value

def attend(d, group):
    shape, p = hs.attn_shape(group, 1, d, 64, "fp8_block"), hs.attn_params(0.1, True)
    kv = hs.PagedKV()
    kv.k_pages, kv.v_pages = on_gpu(np.zeros((2, 64, d), np.uint8)), on_gpu(np.full((2, 64, d), 0x38, np.uint8))
    kv.k_scales = kv.v_scales = on_gpu(np.ones(2, np.float32))
    kv.page_table, kv.seq_lens = on_gpu(np.array([0, 1], np.int32)), on_gpu(np.array([100], np.int32))
    kv.batch, kv.max_blocks, kv.num_pages = 1, 2, 2
    need = hs.hs_workspace_bytes(shape, 1, 2, p)
    out, lse = np.zeros((group, d), np.float32), np.zeros(group, np.float32)
    go, gl = on_gpu(out), on_gpu(lse)
    r = ctypes.byref
    status = hs.library().hs_sparse_paged_decode_attn(
        r(shape), r(kv), on_gpu(np.zeros((group, d), np.uint16)), on_gpu(np.array([0, 1], np.int32)),
        on_gpu(np.array([2], np.int32)), 2, r(p), go, gl, on_gpu(np.zeros(need, np.uint8)), need, None)
    assert status == hs.HS_OK, status
    ok(cu.cuCtxSynchronize())
    ok(cu.cuMemcpyDtoH_v2(out.ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(go), ctypes.c_size_t(out.nbytes)))
    ok(cu.cuMemcpyDtoH_v2(lse.ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(gl), ctypes.c_size_t(lse.nbytes)))
    assert (out == 1).all() and np.abs(lse - math.log(100)).max() < 1e-5  # 4 roundings of a number under 8

ok(cu.cuInit(0))
dev, ctx = ctypes.c_int(), ctypes.c_void_p()
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(ctx), dev))
ok(cu.cuCtxSetCurrent(ctx))
for shape in ((128, 8), (64, 16)):
    attend(*shape)
other = ctypes.c_void_p()
ok(cu.cuCtxCreate_v2(ctypes.byref(other), 0, dev))
for shape in ((128, 8), (64, 16)):
    attend(*shape)
ok(cu.cuCtxDestroy_v2(other))
print("both contexts")
"""


def test_a_second_context_on_the_device():
    """What a launch needs set, once for the device, holds in a context made later."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SECOND_CONTEXT], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "both contexts" in r.stdout, r.stderr


def test_pages_past_4_gib_of_the_pool():
    """Append, summaries and attention on pages whose byte offsets pass 32 bits."""
    from query_aware_sparse_hs_gb300 import hs
    d, block, lens = 128, 64, [130, 64]
    pages = (1 << 32) // (d * block) + 40
    k = torch.empty((pages, block, d), dtype=torch.uint8, device="cuda")
    v = torch.empty((pages, block, d), dtype=torch.uint8, device="cuda")
    ks, vs = torch.empty(pages, device="cuda"), torch.empty(pages, device="cuda")
    table = (pages - 1 - 3 * torch.arange(2 * 3, dtype=torch.int32).view(2, 1, 3)).cuda()
    gl = torch.tensor(lens, dtype=torch.int32).cuda()
    kv = hs.paged_kv(k, v, table, gl, ks, vs)
    shape = hs.attn_shape(4, 1, d, block, "fp8_block")
    rows = torch.randn((sum(lens), 2, d), device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 130, 194], dtype=torch.int32).cuda()
    smin = torch.zeros((2, 1, 3, d), dtype=torch.bfloat16, device="cuda")
    smax = smin.clone()
    hs.hs_append_tokens(shape, kv, hs.append_params(new_offsets=off), rows[:, :1], rows[:, 1:], None, None, smin, smax)
    gl += 1
    one = torch.randn((2, 2, d), device="cuda").to(torch.bfloat16)
    hs.hs_append_tokens(shape, kv, hs.append_params(), one[:, :1], one[:, 1:], None, None, smin, smax)
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)
    c = Cache.__new__(Cache)
    c.lens, c.hkv, c.d, c.block, c.nb, c.kv, c.rng = [131, 65], 1, d, block, [3, 2], kv, np.random.default_rng(1)
    used = table.flatten().long()
    at = {int(p): i for i, p in enumerate(used)}
    c.table = np.array([[[at[int(table[b, 0, j])] for j in range(3)]] for b in range(2)], np.int32)
    c.codes, c.scales = {"k": k[used].cpu().numpy(), "v": v[used].cpu().numpy()}, {"k": ks[used].cpu().numpy(), "v": vs[used].cpu().numpy()}
    for b, L in enumerate(lens):  # what was appended is there
        src = torch.cat([rows[130 * b:130 * b + L], one[b:b + 1]]).double().cpu().numpy()
        for w, i in (("k", 0), ("v", 1)):
            x = c.rows(w, b, 0, range(c.nb[b]))
            s = np.repeat(c.scales[w][c.table[b, 0, :c.nb[b]]], block)[:L + 1, None]
            # half a step of the code, twice where the page's scale grew
            assert (np.abs(x - src[:, i]) <= np.maximum(2.0 ** -4 * np.abs(src[:, i]), 2 * 2.0 ** -10 * s)).all()
    lo, hi = torch.zeros_like(smin), torch.zeros_like(smax)
    hs.hs_build_block_summaries(shape, kv, 0, lo, hi)
    assert torch.equal(lo, smin) and torch.equal(hi, smax)
    q = query(c, 4)
    sel, cnt = chosen(c, 3, None)
    for algo in ("auto", "simt"):
        out, lse = attend(c, q, sel, cnt, algo=algo)
        check_attention(c, q, sel, cnt, out, lse, simt=algo == "simt")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [1, 5, 16, 48, 64, 256])
def test_summaries_match_the_definition(d, block):
    from query_aware_sparse_hs_gb300 import hs
    c = Cache([0, 1, block, block + 1, 5 * block - 1, 777], 2, d, block, seed=block + d)
    shape = hs.attn_shape(4, 2, d, block, "fp8_block")
    for first in (0, 2):
        lo = torch.full((len(c.lens), 2, c.mb, d), 9.0, dtype=torch.bfloat16, device="cuda")
        hi = lo.clone()
        hs.hs_build_block_summaries(shape, c.kv, first, lo, hi)
        for b, n in enumerate(c.nb):
            for h in range(2):
                for j in range(c.mb):
                    got = lo[b, h, j].double().cpu().numpy(), hi[b, h, j].double().cpu().numpy()
                    if j < first or j >= n:
                        assert (got[0] == 9).all() and (got[1] == 9).all()
                        continue
                    x = c.rows("k", b, h, [j])
                    # code times scale in fp32, then outward
                    x32 = x.astype(np.float32)
                    assert np.array_equal(got[0], O.bf16_round_down(x32.min(0))) and np.array_equal(got[1], O.bf16_round_up(x32.max(0)))


def test_summaries_of_extreme_codes_and_scales():
    """Every code that is a number, -0 among them, at scales from 2^-117 to 2^100."""
    from query_aware_sparse_hs_gb300 import hs
    codes = np.array([x for x in range(256) if x & 0x7F != 0x7F], np.uint8)
    c = Cache([64 * 40], 1, 64, 64, seed=2, poison=False)
    c.codes["k"] = codes[c.rng.integers(0, len(codes), c.codes["k"].shape)]
    c.scales["k"] = np.exp2(c.rng.integers(-117, 100, c.pages)).astype(np.float32)
    c.scales["k"][:10] *= 1.37
    c.up()
    lo = torch.zeros((1, 1, c.mb, 64), dtype=torch.bfloat16, device="cuda")
    hi = lo.clone()
    hs.hs_build_block_summaries(hs.attn_shape(1, 1, 64, 64, "fp8_block"), c.kv, 0, lo, hi)
    for j in range(40):
        x = c.rows("k", 0, 0, [j]).astype(np.float32)
        assert np.array_equal(lo[0, 0, j].double().cpu().numpy(), O.bf16_round_down(x.min(0)))
        assert np.array_equal(hi[0, 0, j].double().cpu().numpy(), O.bf16_round_up(x.max(0)))


@pytest.mark.parametrize("d,block", [(128, 64), (128, 16), (64, 32)])
@pytest.mark.parametrize("fuse", [True, False])
def test_prompts_then_decode_steps(d, block, fuse):
    """Prompts appended with rotation, then tokens: append -> selection -> attention, every step against the definition on
    the cache as the append left it."""
    from query_aware_sparse_hs_gb300 import hs
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    hq, hkv, prompts, steps = 16, 2, [5 * block + 3, 20, 9 * block], 5
    batch, dev = len(prompts), "cuda"
    mb = -(-(max(prompts) + steps) // block) + 1
    g = torch.Generator(device=dev).manual_seed(d + block)
    pages = batch * hkv * mb
    k = torch.full((pages, block, d), 0x7F, dtype=torch.uint8, device=dev)
    v = k.clone()
    ks, vs = torch.full((pages,), float("nan"), device=dev), torch.full((pages,), float("nan"), device=dev)
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(batch, hkv, mb)
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    kv = hs.paged_kv(k, v, table, lens, ks, vs)
    dec = SparseDecode(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=block, kv_dtype="fp8_block", batch=batch,
                       max_blocks=mb, sink_tokens=4, window_tokens=block + 1, k_scored=2, out_is_fp32=True, fuse_step=fuse)
    ang = torch.arange(mb * block, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().to(dev)
    off = torch.tensor([0] + list(np.cumsum(prompts)), dtype=torch.int32, device=dev)
    rows = torch.randn((sum(prompts), hq + 2 * hkv, d), generator=g, device=dev).to(torch.bfloat16)
    q_out = torch.empty((sum(prompts), hq, d), dtype=torch.bfloat16, device=dev)
    dec.append_tokens(kv, hs.append_params(cs, new_offsets=off), rows[:, hq:hq + hkv], rows[:, hq + hkv:], rows[:, :hq], q_out)
    one = hs.append_params(cs)
    q1 = torch.empty((batch, hq, d), dtype=torch.bfloat16, device=dev)
    c = Cache.__new__(Cache)
    c.hkv, c.d, c.block, c.table = hkv, d, block, table.cpu().numpy()
    for _ in range(steps):
        lens += 1
        rows = torch.randn((batch, hq + 2 * hkv, d), generator=g, device=dev).to(torch.bfloat16)
        dec.append_tokens(kv, one, rows[:, hq:hq + hkv], rows[:, hq + hkv:], rows[:, :hq], q1)
        dec.step(kv, q1)
        assert hs.hs_get_device_error() == (hs.HS_OK, 0)
        c.lens = lens.tolist()
        c.nb = [-(-n // block) for n in c.lens]
        c.codes, c.scales = {"k": k.cpu().numpy(), "v": v.cpu().numpy()}, {"k": ks.cpu().numpy(), "v": vs.cpu().numpy()}
        sel, cnt = dec.sel.cpu().numpy(), dec.sel_count.cpu().numpy()
        for b in range(batch):
            forced = O.forced_blocks(c.lens[b], block, 4, block + 1)
            for h in range(hkv):
                K = c.rows("k", b, h, range(c.nb[b]))
                smin, smax = O.stored_summaries(*O.block_summaries(K, block), "fp8")
                n = c.nb[b]
                assert np.array_equal(dec.smin[b, h, :n].double().cpu().numpy(), smin)
                assert np.array_equal(dec.smax[b, h, :n].double().cpu().numpy(), smax)
                score = O.bound_scores(q1[b, h * hq // hkv:(h + 1) * hq // hkv].double().cpu().numpy(), smin, smax)[-1]
                assert sel[b, h, :cnt[b, h]].tolist() == O.select_blocks(score, forced, 2)
        check_attention(c, q1, sel, cnt, dec.out, dec.lse)
    # the other step calls: the token appended inside the call
    lens += 1
    new = torch.randn((2, batch, hkv, d), generator=g, device=dev).to(torch.bfloat16)
    a = [t.clone() for t in (k, v, ks, vs, dec.smin, dec.smax)]
    out, lse = (t.clone() for t in dec.step(kv, q1, new_kv=(new[0], new[1])))
    after = [t.clone() for t in (k, v, ks, vs, dec.smin, dec.smax)]
    for dst, src in zip((k, v, ks, vs, dec.smin, dec.smax), a):
        dst.copy_(src)
    dec.append(kv, new[0], new[1])
    dec.select(kv, q1)
    dec.attend(kv, q1)
    for x, y in zip(after + [out, lse], (k, v, ks, vs, dec.smin, dec.smax, dec.out, dec.lse)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    for dst, src in zip((k, v, ks, vs, dec.smin, dec.smax), a):
        dst.copy_(src)
    out2, lse2 = dec.step(kv, q1, new_kv=(new[0], new[1]), reuse=dec)
    assert torch.equal(out2, out) and torch.equal(lse2, lse)
