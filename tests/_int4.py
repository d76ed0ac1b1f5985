"""A 4-bit paged cache for the GPU tests: codes and scales in numpy, what they stand for in 64 bits, and the checks of the
attention over it."""

import math

import numpy as np
import torch

U = 2.0 ** -23  # a rounding of an fp32 sum on the matrix units (truncation counted)


def bf16(x):
    """Nearest bf16 numbers, as float64."""
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.float32).to(torch.bfloat16).double().numpy()


def values(codes, scales):
    """64-bit values of rows: codes [..., D/2] bytes, scales [..., 2, D/32] float64."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.float64) - 8
    s, z = (np.repeat(scales[..., i, :], 32, -1) for i in (0, 1))
    return z + s * c


class Cache:
    """scale: (least, largest) log2 of the scales; offset: deviation of the centres in scales."""

    def __init__(self, lens, hkv, d, block, seed=0, kscale=(-3, -1), vscale=(-3, -1), offset=1.5, poison=True, spare=2):
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
        shape = (self.pages, block)
        self.codes, self.scales = {}, {}
        for w, e in (("k", kscale), ("v", vscale)):
            self.codes[w] = rng.integers(0, 256, shape + (d // 2,), dtype=np.uint8)
            s = bf16(np.exp2(rng.uniform(*e, shape + (1, d // 32))))
            self.scales[w] = np.concatenate([s, bf16(rng.standard_normal(s.shape) * s * offset)], 2)
        if poison:  # rows behind the last token, and pages of nobody, hold NaN
            for b, L in enumerate(lens):
                if L % block:
                    for h in range(hkv):
                        for w in "kv":
                            self.scales[w][self.table[b, h, L // block], L % block:] = np.nan
            for p in order[at:]:
                for w in "kv":
                    self.scales[w][p] = np.nan
        self.up()

    def up(self):
        from query_aware_sparse_hs_gb300 import hs
        self.g = {w: torch.from_numpy(self.codes[w]).cuda() for w in "kv"}
        self.gs = {w: torch.from_numpy(self.scales[w]).cuda().to(torch.bfloat16) for w in "kv"}
        self.gt, self.gl = torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.kv = hs.paged_kv(self.g["k"], self.g["v"], self.gt, self.gl, self.gs["k"], self.gs["v"])

    def part(self, w, b, h, blocks, centres_only=False):
        """64-bit values of the valid tokens of `blocks` (or their centres alone)."""
        out = [np.zeros((0, self.d))]
        for j in blocks:
            n = min(self.block, self.lens[b] - j * self.block)
            p = self.table[b, h, j]
            sc = self.scales[w][p, :n]
            out.append(np.repeat(sc[:, 1], 32, -1) if centres_only else values(self.codes[w][p, :n], sc))
        return np.concatenate(out)


def chosen(c, capacity, keep, shuffle=False):
    """sel and sel_count: `keep` blocks of each (request, kv head) (None: all)."""
    sel = np.full((len(c.lens), c.hkv, capacity), -1, np.int32)
    cnt = np.zeros((len(c.lens), c.hkv), np.int32)
    for b, n in enumerate(c.nb):
        for h in range(c.hkv):
            k = n if keep is None else min(n, keep)
            got = c.rng.permutation(n)[:k]
            sel[b, h, :k] = got if shuffle else np.sort(got)
            cnt[b, h] = k
    return sel, cnt


def query(c, hq, seed=1, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((len(c.lens), hq, c.d), generator=g) * torch.exp2(spread * torch.randn((len(c.lens), hq, 1), generator=g))
    return q.to(torch.bfloat16).cuda()


def attend(c, q, sel, cnt, f32=True, counters=True, algo="auto", max_ctas=0, scale=None, bps=0, lse=True):
    from query_aware_sparse_hs_gb300 import hs
    shape = hs.attn_shape(q.shape[1], c.hkv, c.d, c.block, "int4")
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


def check_attention(c, q, sel, cnt, out, lse, scale=None):
    """Against the definition.  Bounds: a logit is the sum, in fp32, of D exact products of a query's entry and a code of
    0 .. 15, less 8 times the entries' sum, times a scale, and of the centre's product (three terms of 8 bits: 2^-24), so it
    is off by (D + 20) U of the magnitudes' sum, a code counting as 24 scales.  A probability times a V scale enters as two
    f16 terms (2^-21, and absolutely half of f16's smallest step 2^-24 in units of 2^-13 of a reference under twice the
    largest scale or eighth of a centre met, so 2^-37 of that, times a code of 8), times a centre as two bf16 terms (2^-16);
    an output is a sum of T such terms, and one rounding to its type."""
    scale = c.d ** -0.5 if scale is None else scale
    qn, group = q.double().cpu().numpy(), q.shape[1] // c.hkv
    half = 0.0 if out.dtype == torch.float32 else 2.0 ** -8
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(c.lens)):
        for h in range(c.hkv):
            blocks = sel[b, h, :cnt[b, h]]
            K, V = c.part("k", b, h, blocks), c.part("v", b, h, blocks)
            Z, Kz = np.abs(c.part("v", b, h, blocks, True)), np.abs(c.part("k", b, h, blocks, True))
            T = len(K)
            if T:
                ks = np.concatenate([np.repeat(c.scales["k"][c.table[b, h, j], :min(c.block, c.lens[b] - j * c.block), 0], 32, -1)
                                     for j in blocks])
                vs = max(np.max(np.abs(c.scales["v"][c.table[b, h, j], :min(c.block, c.lens[b] - j * c.block)]) * [[1.0], [0.125]])
                         for j in blocks)
            for i in range(h * group, (h + 1) * group):
                if T == 0:
                    assert (got[b, i] == 0).all() and gl[b, i] == -np.inf
                    continue
                s = K @ qn[b, i] * scale
                mags = (24 * ks + Kz) @ np.abs(qn[b, i]) * abs(scale)
                ds = mags.max() * (c.d + 20) * U + 4 * U * np.abs(s).max()
                m = s.max()
                p = np.exp(s - m)
                want, l = (p[:, None] * V).sum(0) / p.sum(), m + math.log(p.sum())
                assert abs(gl[b, i] - l) <= ds + (T + 40) * U + 4 * U * abs(l), (b, i, gl[b, i], l)
                wz = (p[:, None] * Z).sum(0) / p.sum()
                wc = (p[:, None] * (np.abs(V) + Z)).sum(0) / p.sum()  # |s c| at most
                rel = 2 * math.expm1(ds) + (T + 60) * U
                tiny = 8 * 2.0 ** -37 * vs * T / p.sum()
                bound = half * np.abs(want) + (1 + half) * ((rel + 2.0 ** -20) * wc + (rel + 2.0 ** -16) * wz + tiny)
                assert (np.abs(got[b, i] - want) <= bound).all(), (b, i, np.abs(got[b, i] - want).max(), bound.min())
