"""The 4-bit cache: its format, the append into it, attention over it (tensor-core and CUDA-core), its block summaries and
whole decode steps on it, against plain 64-bit arithmetic.  GPU only."""

import numpy as np
import pytest
import torch

from _int4 import Cache, U, attend, bf16, check_attention, chosen, query, values

pytestmark = pytest.mark.gpu


def ok():
    from query_aware_sparse_hs_gb300 import hs
    assert hs.hs_get_device_error() == (hs.HS_OK, 0)


# ---- the format ----------------------------------------------------------------------------------------------------------


def up_bf16(x):
    """The smallest bf16 at or above x >= 0."""
    y = bf16(x)
    bits = torch.from_numpy(y).to(torch.bfloat16).view(torch.int16)
    more = (bits + 1).view(torch.bfloat16).double().numpy()
    return np.where(y < x, more, y)


def quantised(x):
    """(s, z, c) of rows of float64 by the definition, and how far each quotient is from the next border."""
    g = np.clip(x, -2.0 ** 126, 2.0 ** 126).reshape(x.shape[:-1] + (-1, 32))
    lo, hi = g.min(-1), g.max(-1)
    z = bf16((7 * lo + 8 * hi) / 15)
    s = up_bf16(np.maximum((hi - z) / 7, (z - lo) / 8))
    s = np.where(s >= 2.0 ** -116, s, 0.0)
    with np.errstate(invalid="ignore", divide="ignore"):
        quo = np.where(s[..., None] > 0, (g - z[..., None]) / s[..., None], 0.0)
    return s, z, np.clip(np.rint(quo), -8, 7).reshape(x.shape), np.abs(quo - np.floor(quo) - 0.5).reshape(x.shape)


def run_quantise(x, f32):
    from query_aware_sparse_hs_gb300 import hs
    rows, d = x.shape
    src = torch.from_numpy(x).to(torch.float32 if f32 else torch.bfloat16).cuda()
    codes = torch.zeros((rows, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((rows, 2, d // 32), dtype=torch.bfloat16, device="cuda")
    hs.hs_quantize_int4_g32(src, codes, scales)
    return src.double().cpu().numpy(), codes, scales


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows", [1, 7, 1000])
def test_quantise_holds_every_value_within_half_a_step(d, f32, rows):
    rng = np.random.default_rng(d + rows)
    x = rng.standard_normal((rows, d)) * np.exp2(rng.uniform(-20, 20, (rows, 1))) + rng.standard_normal((rows, 1)) * 3
    x[rows // 2] = 2.5  # a group of equal values
    x, codes, scales = run_quantise(x, f32)
    s, z, c, near = quantised(x)
    got_s, got_z = scales.double().cpu().numpy()[:, 0], scales.double().cpu().numpy()[:, 1]
    # fp32 on the way (three roundings) may tip a rounding to bf16, by one step of it
    assert (np.abs(got_z - z) <= 2.0 ** -7 * np.abs(z)).all() and (got_z == z).mean() > 0.99
    assert (np.abs(got_s - s) <= 2.0 ** -6 * s + 2.0 ** -7 * np.abs(z)).all() and (got_s == s).mean() > 0.98
    back = values(codes.cpu().numpy(), scales.double().cpu().numpy())
    step = np.repeat(got_s, 32, -1)
    assert (np.abs(back - x) <= step * (0.5 + 2.0 ** -18) + 2.0 ** -22 * np.abs(x)).all()
    same = np.repeat((got_s == s) & (got_z == z), 32, -1) & (near > 1e-3)
    nibbles = np.stack([codes.cpu().numpy() & 15, codes.cpu().numpy() >> 4], -1).reshape(rows, d).astype(int) - 8
    assert (nibbles == c)[same].all() and same.mean() > 0.9
    assert (back[rows // 2] == 2.5).all()


def test_quantise_of_values_that_are_not_ordinary():
    x = np.tile(np.linspace(-1, 1, 32), (8, 2))
    x[1, 3] = np.nan          # the whole group reads as NaN, the other one is untouched
    x[2, 0] = np.inf          # held as 2^126
    x[3, 5] = -np.inf
    x[4, :32] = 0.0
    x[5, :32] = 2.0 ** -130 * np.arange(32)  # too narrow for a scale: the centre
    x[6, 0], x[6, 1] = 3.0e38, -3.0e38
    x[7, :32] = np.nan
    _, codes, scales = run_quantise(x, True)
    back = values(codes.cpu().numpy(), scales.double().cpu().numpy())
    assert np.isnan(back[1, :32]).all() and np.isnan(back[7, :32]).all()
    for r in range(8):
        assert (np.abs(back[r, 32:] - x[r, 32:]) <= 1 / 14).all()
    for r, i, want in ((2, 0, 2.0 ** 126), (3, 5, -2.0 ** 126), (6, 0, 2.0 ** 126), (6, 1, -2.0 ** 126)):
        assert abs(back[r, i] / want - 1) < 0.06 and np.isfinite(back[r]).all()
    assert (back[4, :32] == 0).all() and (np.abs(back[5, :32]) < 2.0 ** -120).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dequantise_is_the_fp32_value_rounded_once(d, dtype):
    from query_aware_sparse_hs_gb300 import hs
    g = torch.Generator().manual_seed(d)
    codes = torch.randint(0, 256, (501, d // 2), generator=g, dtype=torch.uint8).cuda()
    scales = torch.randn((501, 2, d // 32), generator=g).to(torch.bfloat16).cuda()
    out = torch.zeros((501, d), dtype=dtype, device="cuda")
    hs.hs_dequantize_int4_g32(codes, scales, out)
    want = torch.from_numpy(values(codes.cpu().numpy(), scales.double().cpu().numpy())).float().to(dtype)
    assert torch.equal(out.cpu(), want)


def test_no_rows():
    from query_aware_sparse_hs_gb300 import hs
    e = torch.empty((0, 128), device="cuda")
    c, s = torch.empty((0, 64), dtype=torch.uint8, device="cuda"), torch.empty((0, 2, 4), dtype=torch.bfloat16, device="cuda")
    hs.hs_quantize_int4_g32(e, c, s)
    hs.hs_dequantize_int4_g32(c, s, e)


# ---- append --------------------------------------------------------------------------------------------------------------


def angles(rotary, rows):
    inv = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) / (rotary // 2))
    a = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


APPENDS = {
    # lengths before, new rows, kv heads, group, d, block, rotary, interleaved
    "one_each": ([5, 0, 63, 64, 700], None, 2, 8, 128, 64, 128, False),
    "one_each_d64_part": ([5, 0, 15, 16], None, 3, 2, 64, 16, 16, True),
    "one_each_48_of_64": ([5, 31, 2], None, 1, 1, 64, 32, 48, False),
    "prompts": ([0, 60, 10, 130], [200, 7, 0, 129], 2, 4, 128, 64, 128, False),
    "pages_of_16": ([0, 15, 16], [100, 1, 33], 2, 8, 128, 16, 64, False),
    "pages_of_5_interleaved": ([3, 0], [44, 13], 1, 2, 128, 5, 32, True),
    "d64_rotary_48": ([0, 7], [77, 30], 2, 1, 64, 32, 48, False),
    "pages_of_256": ([200, 0], [300, 513], 1, 8, 128, 256, 128, False),
    "no_rotation": ([0, 20], [40, 3], 2, 2, 64, 48, 0, False),
}


@pytest.mark.parametrize("boxes", [True, False])
@pytest.mark.parametrize("name", list(APPENDS))
def test_append_stores_what_the_quantiser_makes_of_the_rotated_rows(name, boxes):
    """The rotated rows are an f32 cache's, appended from the same values."""
    from query_aware_sparse_hs_gb300 import hs
    old, new, hkv, group, d, block, rotary, inter = APPENDS[name]
    n_new = [1] * len(old) if new is None else new
    lens = [a + n for a, n in zip(old, n_new)]
    c = Cache(lens, hkv, d, block, seed=3, poison=False)
    f = {w: torch.zeros((c.pages, block, d), device="cuda") for w in "kv"}
    wide = hs.paged_kv(f["k"], f["v"], c.gt, c.gl)
    rows = sum(n_new) + (0 if new is None else 3)
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((rows, (group + 2) * hkv, d), generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :group * hkv], qkv[:, group * hkv:(group + 1) * hkv], qkv[:, (group + 1) * hkv:]
    off = None if new is None else torch.tensor(np.concatenate([[0], np.cumsum(n_new)]), dtype=torch.int32).cuda()
    p = hs.append_params(cos_sin=angles(rotary, max(lens) + 1) if rotary else None, interleaved=inter, new_offsets=off)
    shape = hs.attn_shape(group * hkv, hkv, d, block, "int4")
    before = {w: (c.g[w].clone(), c.gs[w].clone()) for w in "kv"}
    smin = smax = None
    if boxes:
        smin = torch.zeros((len(lens), hkv, c.mb, d), dtype=torch.bfloat16, device="cuda")
        smax = torch.zeros_like(smin)
        kept = hs.paged_kv(c.g["k"], c.g["v"], c.gt, torch.tensor(old, dtype=torch.int32).cuda(), c.gs["k"], c.gs["v"])
        hs.hs_build_block_summaries(shape, kept, 0, smin, smax)
    q_out = torch.full_like(q, 7.0).contiguous()
    hs.hs_append_tokens(shape, c.kv, p, k, v, q, q_out, smin, smax)
    ok()
    hs.hs_append_tokens(hs.attn_shape(group * hkv, hkv, d, block, "f32"), wide, p, k.float().contiguous(), v.float().contiguous())
    want = {w: (torch.zeros_like(before[w][0]), torch.zeros_like(before[w][1])) for w in "kv"}
    for w in "kv":
        hs.hs_quantize_int4_g32(f[w], *want[w])
    mine = torch.zeros((c.pages, block), dtype=torch.bool)
    for b, (a, n) in enumerate(zip(old, n_new)):
        for t in range(a, a + n):
            mine[c.table[b, :, t // block], t % block] = True
    mine = mine.cuda()
    for w in "kv":
        for i, x in ((0, c.g[w]), (1, c.gs[w])):
            assert torch.equal(x[mine], want[w][i][mine]) and torch.equal(x[~mine], before[w][i][~mine]), (w, i)
    if new is not None:
        assert (q_out[-3:] == 7).all()  # rows of nobody
    if boxes:
        a, z = torch.zeros_like(smin), torch.zeros_like(smax)
        hs.hs_build_block_summaries(shape, c.kv, 0, a, z)
        assert torch.equal(a, smin) and torch.equal(z, smax)
    ok()


def test_append_token_is_append_tokens_without_rotation():
    from query_aware_sparse_hs_gb300 import hs
    a, b = (Cache([5, 64, 65], 2, 128, 64, seed=2, poison=False) for _ in range(2))
    shape = hs.attn_shape(16, 2, 128, 64, "int4")
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((3, 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    boxes = [torch.zeros((3, 2, a.mb, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    hs.hs_append_token(shape, a.kv, k, v, boxes[0], boxes[1])
    hs.hs_append_tokens(shape, b.kv, hs.append_params(), k, v, smin=boxes[2], smax=boxes[3])
    for w in "kv":
        assert torch.equal(a.g[w], b.g[w]) and torch.equal(a.gs[w], b.gs[w])
    assert torch.equal(boxes[0], boxes[2]) and torch.equal(boxes[1], boxes[3])


def test_a_new_nan_makes_its_group_read_as_nan_and_leaves_the_box():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache([2, 40], 1, 64, 16, seed=2, poison=False)
    shape = hs.attn_shape(2, 1, 64, 16, "int4")
    k = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[0, 0, 7] = float("nan")
    smin = torch.full((2, 1, c.mb, 64), -2.0, dtype=torch.bfloat16, device="cuda")
    smax = torch.full_like(smin, -1.0)
    hs.hs_append_token(shape, c.kv, k, k, smin, smax)
    out = torch.zeros((c.pages, 16, 64), device="cuda")
    hs.hs_dequantize_int4_g32(c.g["k"], c.gs["k"], out)
    row = out[c.table[0, 0, 0], 1]
    assert torch.isnan(row[:32]).all() and (row[32:] == 1).all()
    assert (smax[0, 0, 0, :32] == -1).all() and (smax[0, 0, 0, 32:] == 1).all() and (smin[0, 0, 0] == -2).all()


# ---- attention -----------------------------------------------------------------------------------------------------------

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
    out, lse = attend(c, q, sel, cnt, f32=form != "bf16_out", counters=form != "merge_launch", algo="simt" if form == "simt" else "auto")
    ok()
    check_attention(c, q, sel, cnt, out, lse)


@pytest.mark.parametrize("group,d", [(8, 128), (16, 128), (2, 64), (16, 64)])
def test_bf16_outputs_are_the_fp32_outputs_rounded(group, d):
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
    # hundreds of pairs to a CTA, a long one among them
    c = Cache([1 + 7 * i % 90 for i in range(150)] + [3000], 2, 64, 16, seed=3)
    q = query(c, 4)
    sel, cnt = chosen(c, max(c.nb), None)
    for n in (1, 3, 0):
        for counters in (True, False):
            b, lb = attend(c, q, sel, cnt, max_ctas=n, counters=counters)
            check_attention(c, q, sel, cnt, b, lb)


@pytest.mark.parametrize("vscale,offset", [((-30, 4), 0.0), ((-60, -55), 1.5), ((20, 28), 1.5), ((-3, -1), 40.0)])
def test_v_scales_of_very_different_sizes(vscale, offset):
    c = Cache([700, 64, 2000], 1, 128, 16, seed=4, vscale=vscale, offset=offset)
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt)
    check_attention(c, q, sel, cnt, out, lse)


@pytest.mark.parametrize("vscale", [(-111, -108), (118, 120)])
def test_v_scales_near_the_ends(vscale):
    c = Cache([700, 64, 2000], 1, 64, 16, seed=4, vscale=vscale)
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt)
    assert torch.isfinite(out).all()
    check_attention(c, q, sel, cnt, out, lse)


@pytest.mark.parametrize("top", [1.0, 2.0 ** 60, 2.0 ** -60, 2.0 ** -110])
def test_queries_of_any_size(top):
    """The logits' scale takes the query's size back."""
    c = Cache([100, 7], 1, 128, 16, seed=1)
    q = (query(c, 8).float() * top).to(torch.bfloat16)
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt, scale=0.09 / top)
    check_attention(c, q, sel, cnt, out, lse, scale=0.09 / top)


def test_scales_of_the_logits_that_are_negative_or_zero():
    c = Cache([100, 7], 1, 128, 16, seed=1)
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    for scale in (-0.1, 0.0):
        out, lse = attend(c, q, sel, cnt, scale=scale)
        check_attention(c, q, sel, cnt, out, lse, scale=scale)


@pytest.mark.parametrize("algo", ["auto", "simt"])
def test_a_nan_group_of_v_stays_in_its_channels(algo):
    c = Cache([200, 30], 1, 128, 16, seed=1)
    c.scales["v"][c.table[0, 0, 3], 2, 0, 1] = np.nan
    c.up()
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt, algo=algo)
    assert torch.isnan(out[0, :, 32:64]).all() and torch.isfinite(lse).all()
    c.scales["v"][c.table[0, 0, 3], 2, 0, 1] = 0.0
    rest = [i for i in range(128) if not 32 <= i < 64]
    c.up()
    fine, _ = attend(c, q, sel, cnt, algo=algo)
    assert torch.equal(out[0][:, rest], fine[0][:, rest]) and torch.equal(out[1], fine[1])


def test_a_nan_key_makes_its_heads_nan():
    c = Cache([200, 30], 2, 64, 16, seed=1)
    c.scales["k"][c.table[0, 1, 3], 2, 0, 1] = np.nan
    c.up()
    out, lse = attend(c, query(c, 8), *chosen(c, max(c.nb), None))
    assert torch.isnan(lse[0, 4:]).all() and torch.isnan(out[0, 4:]).all()
    assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all()


def test_a_long_flat_softmax_keeps_its_precision():
    """Queries of 0: every token weighs the same, the output is V's mean, hundreds of times smaller than V."""
    c = Cache([60000], 1, 64, 64, seed=6, offset=0.3)
    q = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda")
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt)
    want = c.part("v", 0, 0, range(c.nb[0])).mean(0)
    assert np.abs(lse.double().cpu().numpy() - np.log(60000)).max() < 1e-4
    # partial sums wander by sqrt(T) of an entry (at most T / 16 of them, each rounded at U of the sum so far)
    step = np.abs(c.scales["v"][..., 0, :][np.isfinite(c.scales["v"][..., 0, :])]).max() * 8
    bound = 60000 / 16 * U * step * np.sqrt(60000) / 60000 + (2.0 ** -16 + 100 * U) * step / np.sqrt(60000) * 4
    assert np.abs(out.double().cpu().numpy()[0] - want).max() <= bound


def test_a_block_selected_twice_counts_twice():
    c = Cache([300], 1, 128, 16, seed=9)
    q = query(c, 8)
    sel = np.full((1, 1, 6), -1, np.int32)
    sel[0, 0, :4] = [2, 2, 5, 18]
    cnt = np.array([[4]], np.int32)
    out, lse = attend(c, q, sel, cnt)
    check_attention(c, q, sel, cnt, out, lse)


def test_what_is_out_of_range_is_reported_and_skipped():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache([300, 100], 1, 128, 16, seed=9)
    q = query(c, 8)
    for algo in ("auto", "simt"):
        sel = np.full((2, 1, 4), -1, np.int32)
        sel[0, 0] = [0, 5, 19, 18]
        sel[1, 0, :2] = [-2147483648, 3]
        cnt = np.array([[9], [2]], np.int32)
        out, lse = attend(c, q, sel, cnt, algo=algo)
        st, bits = hs.hs_get_device_error()
        assert bits == hs.HS_EBIT_CAPACITY | hs.HS_EBIT_BLOCK_RANGE
        fine = np.full((2, 1, 4), -1, np.int32)
        fine[0, 0, :3], fine[1, 0, 0] = [0, 5, 18], 3
        check_attention(c, q, fine, np.array([[3], [1]], np.int32), out, lse)
        bad = c.table.copy()
        bad[0, 0, 5] = c.pages
        c.gt.copy_(torch.from_numpy(bad))
        out, lse = attend(c, q, fine, np.array([[3], [1]], np.int32), algo=algo)
        assert hs.hs_get_device_error()[1] == hs.HS_EBIT_PAGE_RANGE
        c.gt.copy_(torch.from_numpy(c.table))
        fine[0, 0, :3] = [0, 18, -1]
        check_attention(c, q, fine, np.array([[2], [1]], np.int32), out, lse)


def test_pools_past_four_gib():
    """A pool whose rows lie beyond 2^32 bytes."""
    from query_aware_sparse_hs_gb300 import hs
    c = Cache([700, 130], 1, 128, 64, seed=5)
    total = (1 << 32) // (64 * 64) + 64
    far = np.sort(np.random.default_rng(1).choice(np.arange(total - 60, total), c.pages, replace=False))
    g, gs = {}, {}
    for w in "kv":
        g[w] = torch.zeros((total, 64, 64), dtype=torch.uint8, device="cuda")
        gs[w] = torch.zeros((total, 64, 2, 4), dtype=torch.bfloat16, device="cuda")
        g[w][far] = c.g[w]
        gs[w][far] = c.gs[w]
    table = np.where(c.table >= 0, far[np.maximum(c.table, 0)], -1).astype(np.int32)
    q = query(c, 8)
    sel, cnt = chosen(c, max(c.nb), None)
    near, ln = attend(c, q, sel, cnt)
    c.kv = hs.paged_kv(g["k"], g["v"], torch.from_numpy(table).cuda(), c.gl, gs["k"], gs["v"])
    out, lse = attend(c, q, sel, cnt)
    assert torch.equal(out, near) and torch.equal(lse, ln)
    shape = hs.attn_shape(8, 1, 128, 64, "int4")
    a, b = (torch.zeros((2, 1, c.mb, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hs.hs_build_block_summaries(shape, c.kv, 0, a, b)
    c.up()
    x, y = torch.zeros_like(a), torch.zeros_like(b)
    hs.hs_build_block_summaries(shape, c.kv, 0, x, y)
    assert torch.equal(a, x) and torch.equal(b, y)


def test_captured_and_on_another_stream():
    from query_aware_sparse_hs_gb300 import hs
    c = Cache([3000, 900], 2, 128, 64, seed=5)
    q = query(c, 16)
    sel, cnt = chosen(c, max(c.nb), None)
    want, lw = attend(c, q, sel, cnt)
    shape = hs.attn_shape(16, 2, 128, 64, "int4")
    ctr = torch.zeros(4, dtype=torch.int32, device="cuda")
    p = hs.attn_params(128 ** -0.5, True, split_counters=ctr)
    gsel, gcnt = torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()
    ws = torch.empty(hs.hs_workspace_bytes(shape, 2, sel.shape[2], p), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(want), torch.zeros_like(lw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    hs.hs_sparse_paged_decode_attn(shape, c.kv, q, gsel, gcnt, sel.shape[2], p, out, lse, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_sparse_paged_decode_attn(shape, c.kv, q, gsel, gcnt, sel.shape[2], p, out, lse, ws)
    for seed in (7, 8):
        q.copy_(query(c, 16, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        again, la = attend(c, q, sel, cnt)
        assert torch.equal(out, again) and torch.equal(lse, la)


def test_two_calls_at_once_and_the_call_without_a_workspace():
    """Two streams, a workspace and counters each, many times over; and the library's own scratch."""
    from query_aware_sparse_hs_gb300 import hs
    shape = hs.attn_shape(16, 2, 128, 64, "int4")
    jobs = []
    for seed in (1, 2):
        c = Cache([9000, 700, 3000], 2, 128, 64, seed=seed)
        q = query(c, 16, seed=seed)
        sel, cnt = chosen(c, max(c.nb), None)
        want = attend(c, q, sel, cnt)
        ctr = torch.zeros(6, dtype=torch.int32, device="cuda")
        p = hs.attn_params(128 ** -0.5, True, split_counters=ctr)
        ws = torch.empty(hs.hs_workspace_bytes(shape, 3, sel.shape[2], p), dtype=torch.uint8, device="cuda")
        jobs.append((c, q, torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda(), p, ws, torch.zeros_like(want[0]),
                     torch.zeros_like(want[1]), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, sel, cnt, p, ws, out, lse, _, stream in jobs:
            hs.hs_sparse_paged_decode_attn(shape, c.kv, q, sel, cnt, sel.shape[2], p, out, lse, ws, stream=stream)
    torch.cuda.synchronize()
    for c, q, sel, cnt, p, ws, out, lse, want, _ in jobs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        out.fill_(float("nan"))
        hs.hs_sparse_paged_decode_attn_noalloc(shape, c.kv, q, sel, cnt, sel.shape[2], p, out, lse)
        assert torch.equal(out, want[0])
    ok()


# ---- summaries -----------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("lens,hkv,d,block,first", [
    ([1], 1, 128, 64, 0), ([0, 500, 0, 33, 0], 2, 128, 16, 0), ([700, 3, 65], 2, 64, 64, 2), ([44, 201], 3, 64, 5, 0),
    ([1000, 255], 1, 128, 256, 1), ([5, 40], 1, 64, 1, 0), ([1 + 7 * i % 90 for i in range(300)], 2, 128, 48, 0)])
def test_summaries_are_the_outward_rounded_box(lens, hkv, d, block, first):
    from query_aware_sparse_hs_gb300 import hs
    c = Cache(lens, hkv, d, block, seed=d + block)
    shape = hs.attn_shape(hkv, hkv, d, block, "int4")
    lo = torch.full((len(lens), hkv, c.mb, d), 9.0, dtype=torch.bfloat16, device="cuda")
    hi = torch.full_like(lo, 9.0)
    hs.hs_build_block_summaries(shape, c.kv, first, lo, hi)
    ok()
    a, z = lo.double().cpu().numpy(), hi.double().cpu().numpy()
    for b in range(len(lens)):
        for h in range(hkv):
            assert (a[b, h, c.nb[b]:] == 9).all() and (a[b, h, :first] == 9).all()
            for j in range(first, c.nb[b]):
                x = c.part("k", b, h, [j]).astype(np.float32).astype(np.float64)
                mn, mx = x.min(0), x.max(0)
                down, up = bf16(mn), bf16(mx)
                assert (a[b, h, j] <= mn).all() and (z[b, h, j] >= mx).all()
                assert ((a[b, h, j] == down) | (down > mn)).all() and ((z[b, h, j] == up) | (up < mx)).all()
                assert (mn - a[b, h, j] <= 2.0 ** -7 * np.abs(mn)).all() and (z[b, h, j] - mx <= 2.0 ** -7 * np.abs(mx)).all()


# ---- decode steps --------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("hkv,group,d,block", [(2, 8, 128, 64), (1, 16, 64, 16), (4, 2, 128, 16)])
def test_a_decode_step_is_its_calls_in_order(hkv, group, d, block):
    from query_aware_sparse_hs_gb300 import hs
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    lens = [900, 40, 1]
    got = []
    for whole in (True, False):
        c = Cache(lens, hkv, d, block, seed=4, poison=False)
        dec = SparseDecode(num_q_heads=group * hkv, num_kv_heads=hkv, head_dim=d, block_size=block, kv_dtype="int4", batch=3,
                           max_blocks=c.mb, sink_tokens=4, window_tokens=block, k_scored=5, out_is_fp32=True)
        g = torch.Generator().manual_seed(2)
        k, v = (torch.randn((3, hkv, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        q = query(c, group * hkv)
        dec.smin.zero_()  # (blocks that no request has are not written)
        dec.smax.zero_()
        dec.build_summaries(c.kv)
        if whole:
            dec.step(c.kv, q, new_kv=(k, v))
        else:
            dec.append(c.kv, k, v)
            dec.select(c.kv, q)
            dec.attend(c.kv, q)
        ok()
        got.append((dec.out.clone(), dec.lse.clone(), dec.sel.clone(), c.g["k"].clone(), dec.smin.clone()))
        if whole:
            again, _ = dec.step(c.kv, q, new_kv=(k, v), reuse=dec)
            assert torch.equal(again, got[0][0])
        for w in "kv":  # against the definition, over the selection that was made
            c.codes[w], c.scales[w] = c.g[w].cpu().numpy(), c.gs[w].double().cpu().numpy()
        check_attention(c, q, dec.sel.cpu().numpy(), dec.sel_count.cpu().numpy(), dec.out, dec.lse)
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("top", [126, 118, 110, 100, 20])
@pytest.mark.parametrize("group,d", [(8, 128), (16, 64)])
@pytest.mark.parametrize("max_ctas", [0, 1])
def test_large_centres_under_many_small_probabilities(group, d, top, max_ctas):
    """Every token has the same centres, and codes of 0: the output is the centres, whatever the probabilities are.  They enter
    to 16 bits, or absolutely within 2^-146 of the largest V scale, 2^top, times as many as there are over their sum; the sums
    are off by a rounding for each token.  (Every 500th token has 1, the others 2^-8.0 or 2^-9.6.)"""
    T = 12000
    c = Cache([T], 1, d, 64, seed=9)
    c.scales["k"][:, :, 0], c.scales["k"][:, :, 1] = 1.6015625, 0.0
    codes = c.rng.integers(9, 11, T + 32).astype(np.uint8)  # of channel 0: c + 8
    codes[7::500] = 15
    c.codes["k"][:] = c.codes["v"][:] = 0x88
    c.codes["k"][c.table[0, 0, :c.nb[0]], :, 0] = 0x80 | codes.reshape(-1, 64)
    z = bf16((1 + c.rng.random(d // 32)) * 2.0 ** (top - 1) * c.rng.choice([-1.0, 1.0], d // 32))
    c.scales["v"][:, :, 0], c.scales["v"][:, :, 1] = 2.0 ** top, z
    c.up()
    q = torch.zeros((1, group, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    sel, cnt = chosen(c, max(c.nb), None)
    out, lse = attend(c, q, sel, cnt, scale=float(np.log(2)), max_ctas=max_ctas)
    ok()
    s = (codes[:T] - 8.0) * 1.6015625  # logits, in log2 units
    total = np.exp2(s - s.max()).sum()
    bound = 2.0 ** -16 + (T + 60) * U + 2.0 ** (top - 146) * T / total
    off = np.abs(out[0].double().cpu().numpy() / np.repeat(z, 32) - 1.0).max()
    assert off <= bound, (off, bound)
    assert np.abs(lse.cpu().numpy() - (s.max() + np.log2(total)) * np.log(2)).max() < 1e-3
