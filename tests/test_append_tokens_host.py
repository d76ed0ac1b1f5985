"""Refusals of hs_append_tokens and of the block-scaled e4m3 cache, answered on the host before anything is launched, and
the binding's own checks of shapes and types.  CPU only: the addresses are never followed."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

P = 0x10000


def _args(hs, kind="bf16", batch=2, d=128, **kw):
    shape = hs.attn_shape(8, 2, d, 16, kind)
    kv = hs.PagedKV()
    kv.k_pages = kv.v_pages = kv.page_table = kv.seq_lens = P
    if kind.startswith("fp8"):
        kv.k_scales = kv.v_scales = P
    kv.batch, kv.max_blocks, kv.num_pages = batch, 4, 16
    p = hs.AppendParams()
    p.new_offsets, p.positions, p.cos_sin = P, None, P
    p.table_rows, p.rotary_dim, p.interleaved = 64, d, 0
    a = dict(shape=shape, kv=kv, params=p, rows=5, q=P, q_stride=8 * d, q_out=P + 16, q_out_stride=8 * d, k=P, k_stride=2 * d,
             v=P, v_stride=2 * d, smin=P, smax=P)
    for k, v in kw.items():
        if hasattr(p, k):
            setattr(p, k, v)
        elif k in a:
            a[k] = v
        else:
            setattr(kv, k, v)
    return a


def _call(hs, a):
    ref = [ctypes.byref(a["shape"]), None if a["kv"] is None else ctypes.byref(a["kv"]),
           None if a["params"] is None else ctypes.byref(a["params"])]
    rest = [a[k] for k in ("rows", "q", "q_stride", "q_out", "q_out_stride", "k", "k_stride", "v", "v_stride", "smin", "smax")]
    return hs.library().hs_append_tokens(*ref, *rest, None)


@pytest.mark.parametrize("change", [
    {"kv": None}, {"params": None}, {"rows": -1}, {"rows": 1 << 31}, {"k": None}, {"v": None},
    {"q": None}, {"q_out": None},                      # one of the two
    {"smin": None}, {"smax": None},                    # one of the two
    {"k": P + 8}, {"v": P + 2}, {"q": P + 8}, {"q_out": P + 4}, {"smin": P + 8}, {"smax": P + 8},  # alignment
    {"k_stride": 2 * 128 - 8}, {"v_stride": 0}, {"q_stride": 8 * 128 - 8}, {"q_out_stride": 100},  # rows that overlap
    {"k_stride": 2 * 128 + 4}, {"q_stride": 8 * 128 + 1},  # rows off 16 bytes
    {"q_out": P, "q_out_stride": 9 * 128},             # in place with another stride
    {"new_offsets": None},                             # rows is not the batch
    {"new_offsets": P + 2}, {"positions": P + 1}, {"cos_sin": None}, {"cos_sin": P + 8},
    {"rotary_dim": -16}, {"rotary_dim": 144}, {"table_rows": -1},
    {"num_pages": -1}, {"max_blocks": 0}, {"batch": -1}, {"page_table": None}, {"seq_lens": None}, {"v_pages": None},
])
def test_invalid_arguments(change):
    from query_aware_sparse_hs_gb300 import hs
    assert _call(hs, _args(hs, **change)) == hs.HS_ERR_INVALID_ARG


def test_unsupported_rotations_and_sizes():
    from query_aware_sparse_hs_gb300 import hs
    assert _call(hs, _args(hs, rotary_dim=24)) == hs.HS_ERR_UNSUPPORTED
    assert _call(hs, _args(hs, rotary_dim=8)) == hs.HS_ERR_UNSUPPORTED
    a = _args(hs)
    a["shape"] = hs.attn_shape(8, 2, 96, 16, "bf16")
    assert _call(hs, a) == hs.HS_ERR_UNSUPPORTED
    # more CTAs than a grid holds
    a = _args(hs, rows=(1 << 31) - 1)
    a["shape"] = hs.attn_shape(64, 64, 128, 1, "bf16")
    a.update(k_stride=64 * 128, v_stride=64 * 128, q_stride=64 * 128, q_out_stride=64 * 128)
    assert _call(hs, a) == hs.HS_ERR_UNSUPPORTED


def test_block_scaled_cache_needs_its_scales_and_has_no_hot_buffer():
    from query_aware_sparse_hs_gb300 import hs
    assert hs.KV_DTYPES["fp8_block"] == 3
    assert _call(hs, _args(hs, "fp8_block", k_scales=None)) == hs.HS_ERR_INVALID_ARG
    assert _call(hs, _args(hs, "fp8_block", v_scales=None)) == hs.HS_ERR_INVALID_ARG
    assert _call(hs, _args(hs, "fp8_block", k_scales=P + 2)) == hs.HS_ERR_INVALID_ARG
    shape = hs.attn_shape(8, 2, 128, 16, "fp8_block")
    hb = hs.HotBuffer()
    for f in ("page_table", "slot_owner", "last_used", "k_slots", "v_slots", "k_slot_scales", "v_slot_scales", "host_k",
              "host_v", "host_k_scales", "host_v_scales"):
        setattr(hb, f, P)
    hb.batch, hb.max_blocks, hb.slots_per_stream = 1, 4, 4
    assert hs.library().hs_swapin_misses(ctypes.byref(shape), ctypes.byref(hb), P, P, 4, 0, None, None) == hs.HS_ERR_UNSUPPORTED
    bad = hs.attn_shape(8, 2, 128, 16, 4)
    assert hs.library().hs_build_block_summaries(ctypes.byref(bad), None, 0, None, None, None) == hs.HS_ERR_INVALID_ARG


def test_workspace_of_the_block_scaled_attention_does_not_grow_with_the_batch():
    from query_aware_sparse_hs_gb300 import hs
    p = hs.attn_params(0.1)
    small = hs.hs_workspace_bytes(hs.attn_shape(32, 4, 128, 64, "fp8_block"), 1, 1, p)
    assert small > 0
    # two partial results of a group for each CTA; the CUDA-core kernel's uniform splits may need more
    p = hs.attn_params(0.1, blocks_per_split=2048)
    assert hs.hs_workspace_bytes(hs.attn_shape(32, 4, 128, 64, "fp8_block"), 8, 2048, p) == small


def test_geometry_queries_of_the_block_scaled_cache():
    from query_aware_sparse_hs_gb300 import hs
    shape, p = hs.attn_shape(32, 4, 128, 64, "fp8_block"), hs.attn_params(0.1)
    assert hs.hs_attn_geometry(shape, 8, 64, p) == (0, 0)
    assert hs.hs_score_select_attend_fused(shape, 8, 512, 64, p) in (0, -1)  # (-1: no device here)
    assert hs.hs_score_select_attend_workspace_bytes(shape, 8, 512, 64, p) == \
        hs.hs_select_workspace_bytes(shape, 8, 512) + hs.hs_workspace_bytes(shape, 8, 64, p)


def test_the_binding_checks_shapes_and_types():
    from query_aware_sparse_hs_gb300 import hs
    shape = hs.attn_shape(8, 2, 64, 16, "bf16")
    kv = hs.PagedKV()
    kv.batch = 3
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((5, 8, 64), dtype=torch.bfloat16)
    off = torch.zeros(4, dtype=torch.int32)
    ok = hs.append_params(torch.zeros((10, 64)), new_offsets=off)
    assert ok.rotary_dim == 64 and ok.table_rows == 10
    for bad in ({"new_k": k.float()}, {"new_k": k[:4]}, {"new_k": k.transpose(1, 2)}, {"q": q, "q_out": None},
                {"q": q[:, :4], "q_out": q[:, :4]}, {"q": q.float(), "q_out": q}):
        args = dict(new_k=k, new_v=k, q=q, q_out=q.clone())
        args.update(bad)
        with pytest.raises(ValueError):
            hs.hs_append_tokens(shape, kv, ok, **args)
    with pytest.raises(ValueError):
        hs.append_params(torch.zeros((10, 64), dtype=torch.float64))
    with pytest.raises(ValueError):
        hs.append_params(torch.zeros((10, 64)), rotary_dim=32)
    with pytest.raises(ValueError):
        hs.append_params(new_offsets=off.long())
    with pytest.raises(ValueError):  # offsets of another batch
        hs.hs_append_tokens(shape, kv, hs.append_params(new_offsets=off[:3]), k, k)
    with pytest.raises(ValueError):  # fewer positions than rows
        hs.hs_append_tokens(shape, kv, hs.append_params(new_offsets=off, positions=off), k, k)


def test_the_binding_loads_on_a_torch_without_cuda():
    """Such a torch lacks the names that the short ways to the current device and stream take."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from query_aware_sparse_hs_gb300 import hs
shape, kv = hs.attn_shape(8, 2, 64, 16, "bf16"), hs.PagedKV()
kv.batch = 3
rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
try:
    hs.hs_append_tokens(shape, kv, hs.append_params(), rows, rows)
except ValueError as e:
    print("refused:", e)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "on the current device" in r.stdout, r.stderr


def test_addresses_may_be_of_a_subclass_of_int():
    from query_aware_sparse_hs_gb300 import hs

    class Address(int):
        pass

    assert hs.select_params(0, 0, 1, 1, 0.5, Address(P)).score_history == P
    assert hs.attn_params(0.1, split_counters=Address(P)).split_counters == P


def test_params_filled_in_by_hand_are_taken():
    """With addresses in them, as the structures of the other calls: nothing but what the library checks."""
    from query_aware_sparse_hs_gb300 import hs
    shape, kv = hs.attn_shape(8, 2, 64, 16, "bf16"), hs.PagedKV()
    kv.batch = 3
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    p = hs.AppendParams()
    p.new_offsets, p.table_rows = P, 0
    with pytest.raises(ValueError, match="on the current device"):  # the rows are not on a GPU
        hs.hs_append_tokens(shape, kv, p, rows, rows)
    assert p._requests is None and p._rows is None
