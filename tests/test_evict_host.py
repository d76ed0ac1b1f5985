"""Refusals of the 4-bit cache, the accumulated weights and the eviction, before anything is launched.  CPU only."""

import ctypes

import pytest
import torch

P = 0x10000  # an aligned address that nothing reads


def kv(hs, batch=2, mb=8, pages=16, **more):
    k = hs.PagedKV()
    k.k_pages = k.v_pages = k.k_scales = k.v_scales = k.page_table = k.seq_lens = P
    k.batch, k.max_blocks, k.num_pages = batch, mb, pages
    for name, value in more.items():
        setattr(k, name, value)
    return k


def ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.fixture
def hs():
    from query_aware_sparse_hs_gb300 import hs
    return hs


def test_quantise_and_dequantise(hs):
    lib = hs.library()
    for call in (lambda s, r, d, c, z: lib.hs_quantize_int4_g32(s, 0, r, d, c, z, None),
                 lambda s, r, d, c, z: lib.hs_dequantize_int4_g32(c, z, r, d, s, 0, None)):
        assert call(None, 4, 128, P, P) == hs.HS_ERR_INVALID_ARG
        assert call(P, 4, 128, None, P) == hs.HS_ERR_INVALID_ARG
        assert call(P, 4, 128, P, None) == hs.HS_ERR_INVALID_ARG
        assert call(P, -1, 128, P, P) == hs.HS_ERR_INVALID_ARG
        assert call(P + 8, 4, 128, P, P) == hs.HS_ERR_INVALID_ARG
        assert call(P, 4, 128, P + 2, P) == hs.HS_ERR_INVALID_ARG
        assert call(P, 4, 128, P, P + 2) == hs.HS_ERR_INVALID_ARG
        assert call(P, 4, 96, P, P) == hs.HS_ERR_UNSUPPORTED
        assert call(P, 1 << 40, 128, P, P) == hs.HS_ERR_UNSUPPORTED
    x = torch.zeros((4, 128))
    c, s = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 2, 4), dtype=torch.bfloat16)
    for bad in ((x.half(), c, s), (x, c.int(), s), (x, c, s.float()), (x, c[:3], s), (x, c, s[:3]), (x, c.view(8, 32), s)):
        with pytest.raises(ValueError):
            hs.hs_quantize_int4_g32(*bad)
        with pytest.raises(ValueError):
            hs.hs_dequantize_int4_g32(bad[1], bad[2], bad[0])
    with pytest.raises(ValueError, match="current CUDA device"):  # right, but on the host
        hs.hs_quantize_int4_g32(x, c, s)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_dequantize_int4_g32(c, s, x)


def test_a_4_bit_cache(hs):
    lib = hs.library()
    shape = hs.attn_shape(16, 2, 128, 64, "int4")
    for bad in (kv(hs, k_scales=None), kv(hs, k_scales=P + 8), kv(hs, k_pages=P + 8), kv(hs, num_pages=-1)):
        assert lib.hs_build_block_summaries(ref(shape), ref(bad), 0, P, P, None) == hs.HS_ERR_INVALID_ARG
    for bad in (kv(hs, v_scales=None), kv(hs, v_scales=P + 4), kv(hs, v_pages=None)):
        assert lib.hs_append_token(ref(shape), ref(bad), P, P, P, P, None) == hs.HS_ERR_INVALID_ARG
        params = hs.attn_params(0.1)
        assert lib.hs_sparse_paged_decode_attn(ref(shape), ref(bad), P, P, P, 4, ref(params), P, None, P, 1 << 30,
                                               None) == hs.HS_ERR_INVALID_ARG
    # no host pool of 4-bit pages
    hb = hs.HotBuffer()
    for f in ("page_table", "slot_owner", "last_used", "k_slots", "v_slots", "host_k", "host_v", "k_slot_scales", "v_slot_scales",
              "host_k_scales", "host_v_scales"):
        setattr(hb, f, P)
    hb.batch, hb.max_blocks, hb.slots_per_stream = 2, 8, 4
    assert lib.hs_swapin_misses(ref(shape), ref(hb), P, P, 4, 0, None, None) == hs.HS_ERR_UNSUPPORTED
    assert lib.hs_swapin_copy(ref(shape), ref(hb), P, P, 4, 0, None, None) == hs.HS_ERR_UNSUPPORTED
    assert hs.hs_workspace_bytes(shape, 2, 4, hs.attn_params(0.1)) > 0
    past = hs.AttnShape(16, 2, 128, 64, 5)
    assert lib.hs_build_block_summaries(ref(past), ref(kv(hs)), 0, P, P, None) == hs.HS_ERR_INVALID_ARG


def test_accumulated_weights(hs):
    lib = hs.library()
    shape = hs.attn_shape(16, 2, 128, 64, "bf16")

    def call(s=shape, c=None, q=P, lse=P, sel=P, cnt=P, cap=4, w=P):
        return lib.hs_accumulate_attn_weights(ref(s), ref(kv(hs) if c is None else c), q, lse, sel, cnt, cap, 0.1, w, None)

    for bad in ({"q": None}, {"lse": None}, {"sel": None}, {"cnt": None}, {"w": None}, {"cap": 0}, {"q": P + 8}, {"lse": P + 2},
                {"sel": P + 1}, {"cnt": P + 2}, {"w": P + 2}, {"c": kv(hs, k_pages=None)}, {"c": kv(hs, batch=-1)}, {"s": None}):
        assert call(**bad) == hs.HS_ERR_INVALID_ARG, bad
    assert call(s=hs.attn_shape(16, 2, 96, 64, "bf16")) == hs.HS_ERR_UNSUPPORTED
    assert call(c=kv(hs, batch=1 << 30)) == hs.HS_ERR_UNSUPPORTED
    k = kv(hs)
    lse, w = torch.zeros((2, 16)), torch.zeros((2, 2, 8 * 64))
    q, sel, cnt = torch.zeros((2, 16, 128), dtype=torch.bfloat16), torch.zeros((2, 2, 4), dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32)
    for bad in ((q, lse.half(), sel, cnt, w), (q, lse, sel, cnt, w.half()), (q, lse, sel, cnt, w[:, :, 1:]), (q.float(), lse, sel, cnt, w),
                (q[:1], lse, sel, cnt, w), (q, lse[:1], sel, cnt, w), (q, lse, sel.long(), cnt, w), (q, lse, sel[:, :, :3], cnt, w),
                (q, lse, sel, cnt[:1], w), (q, lse, sel, cnt.float(), w)):
        with pytest.raises(ValueError, match="lse"):
            hs.hs_accumulate_attn_weights(shape, k, *bad[:4], 4, 0.1, bad[4])
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_accumulate_attn_weights(shape, k, q, lse, sel, cnt, 4, 0.1, w)


def test_eviction(hs):
    lib = hs.library()
    shape = hs.attn_shape(16, 2, 128, 64, "bf16")

    def call(s=shape, c=None, d=None, p=(100, 4, 32), w=P, dw=P + 64, kept=P):
        params = None if p is None else hs.evict_params(*p)
        return lib.hs_evict_tokens(ref(s), ref(kv(hs) if c is None else c), ref(kv(hs) if d is None else d), ref(params), w, dw, kept, None)

    for bad in ({"p": None}, {"w": None}, {"kept": None}, {"dw": P}, {"w": P + 2}, {"dw": P + 66}, {"kept": P + 1}, {"p": (0, 0, 0)},
                {"p": (-1, 0, 0)}, {"p": (100, -1, 0)}, {"p": (100, 0, -1)}, {"p": (100, 60, 41)}, {"p": (8 * 64 + 1, 0, 0)},
                {"p": (100, 2147483647, 2147483647)}, {"d": kv(hs, batch=3)}, {"c": kv(hs, v_pages=None)}, {"d": kv(hs, k_pages=None)},
                {"d": kv(hs, v_pages=P + 4)}, {"s": None}):
        assert call(**bad) == hs.HS_ERR_INVALID_ARG, bad
    assert call(s=hs.attn_shape(16, 2, 128, 64, "fp8_block")) == hs.HS_ERR_UNSUPPORTED
    big = dict(batch=1 << 20, mb=1 << 20)
    assert call(c=kv(hs, **big), d=kv(hs, **big), p=(1 << 25, 0, 0)) == hs.HS_ERR_UNSUPPORTED
    k = kv(hs)
    w, kept = torch.zeros((2, 2, 8 * 64)), torch.zeros((2, 2, 100), dtype=torch.int32)
    p = hs.evict_params(100)
    for bad in ((w.double(), w.clone(), kept), (w[:, :1], w.clone(), kept), (w, w[:, :1].clone(), kept), (w, w.half(), kept),
                (w, None, kept.long()), (w, None, kept[:, :, 1:])):
        with pytest.raises(ValueError, match="must be"):
            hs.hs_evict_tokens(shape, k, k, p, *bad)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_evict_tokens(shape, k, k, p, w, w.clone(), kept)


def test_the_driver_refuses_a_cache_of_another_length(hs, monkeypatch):
    from query_aware_sparse_hs_gb300.decode import SparseDecode
    dec = SparseDecode.__new__(SparseDecode)
    dec.max_blocks = 9
    with pytest.raises(ValueError):
        dec.evict(kv(hs), kv(hs), hs.evict_params(10), None, None, None)


def test_eviction_of_requests_whose_places_pass_31_bits(hs):
    """Places are counted in 32 bits, some thousands past the last one: a table of 2^31 - 2^14 places or more is refused, and so
    is such a budget."""
    lib = hs.library()
    most = 2 ** 31 - 2 ** 14

    def call(places, budget, room, block):
        shape = hs.attn_shape(8, 1, 64, block, "int4")
        c, d = kv(hs, batch=1, mb=places // block), kv(hs, batch=1, mb=room // block)
        return lib.hs_evict_tokens(ref(shape), ref(c), ref(d), ref(hs.evict_params(budget)), P, None, P, None)

    for block in (1, 64, 256):
        assert call(most, 4096, 4096, block) == hs.HS_ERR_UNSUPPORTED
        assert call(2 ** 31 - block, 4096, 4096, block) == hs.HS_ERR_UNSUPPORTED
        assert call(65536, most, 2 ** 31 - block, block) == hs.HS_ERR_UNSUPPORTED
        assert call(65536, 2 ** 31 - 256, 2 ** 31 - block, block) == hs.HS_ERR_UNSUPPORTED


def driver(monkeypatch, hs, **more):
    """A decoder without device buffers, the library's calls noted and not made."""
    from query_aware_sparse_hs_gb300 import decode
    calls = []
    monkeypatch.setattr(decode.hs, "hs_evict_tokens", lambda *a: calls.append("evict"))
    monkeypatch.setattr(decode.hs, "hs_build_block_summaries", lambda *a: calls.append("summaries"))
    dec = decode.SparseDecode.__new__(decode.SparseDecode)
    dec.shape, dec.batch, dec.max_blocks, dec.smin, dec.smax = hs.attn_shape(8, 2, 128, 16, "int4"), 3, 4, None, None
    for name, value in more.items():
        setattr(dec, name, value)
    return dec, calls


def test_the_driver_forgets_the_scores_of_requests_that_were_cut(hs, monkeypatch):
    """Blocks of a cut request hold other tokens: their smoothed scores are not those of the new ones.  A request shorter than
    the budget keeps its blocks and their scores."""
    history = torch.arange(24.0).view(3, 2, 4) + 1
    before = history.clone()
    dec, calls = driver(monkeypatch, hs, score_history=history)
    kept = torch.tensor([[0, 1, 2, 3, 4], [0, 1, 2, -1, -1], [0, 7, 8, 30, 31]], dtype=torch.int32)[:, None, :].repeat(1, 2, 1)
    c = kv(hs, batch=3, mb=4)
    dec.evict(c, c, hs.evict_params(5, 1, 1), None, None, kept)
    assert calls == ["evict", "summaries"]
    assert dec.score_history is history and history[0].isnan().all() and history[2].isnan().all()
    assert torch.equal(history[1], before[1])
    dec.score_history = None  # no smoothing
    dec.evict(c, c, hs.evict_params(5, 1, 1), None, None, kept)


def test_the_driver_starts_the_weights_of_tokens_to_come_at_0(hs, monkeypatch):
    """Two weight buffers that take turns: the one written now still holds what was there two cuts ago, behind the new length."""
    dec, _ = driver(monkeypatch, hs, score_history=None)
    kept = torch.tensor([[0, 1, 2, 3, 4], [0, 1, 2, -1, -1], [-1] * 5], dtype=torch.int32)[:, None, :].repeat(1, 2, 1)
    w = torch.rand(3, 2, 64) + 1
    want = w.clone()
    for b, n in enumerate((5, 3, 0)):
        want[b, :, n:] = 0.0
    c = kv(hs, batch=3, mb=4)
    dec.evict(c, c, hs.evict_params(5), None, w, kept)
    assert torch.equal(w, want)
    dec.evict(c, c, hs.evict_params(5), None, None, kept)  # none wanted


def test_the_driver_with_a_batch_of_none(hs, monkeypatch):
    dec, calls = driver(monkeypatch, hs, score_history=torch.ones(3, 2, 4))
    c = kv(hs, batch=0, mb=4)
    dec.evict(c, c, hs.evict_params(5), None, torch.ones(0, 2, 64), torch.zeros((0, 2, 5), dtype=torch.int32))
    assert calls == ["evict", "summaries"] and (dec.score_history == 1).all()


def test_attention_whose_lse_is_no_float_address(hs):
    lib, params = hs.library(), hs.attn_params(0.1)
    for kind in ("int4", "bf16", "fp8", "fp8_block", "f32"):
        shape = hs.attn_shape(16, 2, 128, 64, kind)
        for off in (1, 2, 3):
            assert lib.hs_sparse_paged_decode_attn(ref(shape), ref(kv(hs)), P, P, P, 4, ref(params), P, P + off, P, 1 << 30,
                                                   None) == hs.HS_ERR_INVALID_ARG
