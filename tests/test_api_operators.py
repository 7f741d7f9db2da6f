"""Host-side refusals of windowed plans, trees and the quantised cache (no GPU needed): what the library
says before it touches a device, and what the binding says before an address reaches the library."""
import ctypes

import pytest
import torch

from two_tower_block_b200 import ops
from two_tower_block_b200.ops import Shape

BAD = ops.TT_ERR_INVALID_ARG


def desc(**kw):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=4, ctx_capacity=32, seq_len=0, scale=0.0,
             kernel=0, num_ctas=0, flags=0, wait_timeout_us=0)
    return ops.Desc(**{**d, **kw})


@pytest.mark.parametrize("window,sinks", [(-1, 0), (8, -1), (0, 4)])
def test_windows_are_checked_before_the_device(window, sinks):
    h = ctypes.c_void_p()
    assert ops.lib().tt_block_attn_plan_window(ctypes.byref(desc()), window, sinks, 0, ctypes.byref(h)) == BAD
    assert b"window" in ops.lib().tt_last_error_detail()
    assert ops.lib().tt_block_attn_plan_window(None, 8, 0, 0, ctypes.byref(h)) == BAD


def test_calls_without_a_plan_or_a_cache():
    L = ops.lib()
    cache = ops.MxCacheDesc(16, 16, 16, 16, None, 0, 0, 0)
    ref = ctypes.byref(cache)
    assert L.tt_block_attn_tree(None, *[None] * 10) == BAD
    assert L.tt_block_attn_tree_paged(None, None, None, None, None, 1, 24, 1, *[None] * 7) == BAD   # page size 24
    assert L.tt_block_attn_mx(None, None, None, *[None] * 7) == BAD
    assert L.tt_block_attn_mx(None, None, ref, *[None] * 7) == BAD
    assert L.tt_kv_append_mx(None, None, None, 1, None, ref, None, 1, None) == BAD
    assert L.tt_kv_append_mx(None, None, None, 1, None, None, None, 1, None) == BAD
    assert L.tt_kv_read_mx(None, ref, None, None, 1, None, None, None) == BAD
    no_scales = ops.MxCacheDesc(16, 16, None, 16, None, 0, 0, 0)
    assert L.tt_block_attn_mx(None, None, ctypes.byref(no_scales), *[None] * 7) == BAD
    bad_page = ops.MxCacheDesc(16, 16, 16, 16, 4, 1, 8, 1)
    assert L.tt_kv_read_mx(None, ctypes.byref(bad_page), None, None, 1, None, None, None) == BAD
    assert b"page_size" in L.tt_last_error_detail()


def shape_only_plan(cap=32):
    plan = ops.Plan.__new__(ops.Plan)
    plan.shape, plan.device, plan._h = Shape(2, 8, 2, 64, 4, cap, 0), 0, None
    return plan


def decode_inputs(cap=32):
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    kb = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    kc = torch.zeros(2, 2, cap, 64, dtype=torch.bfloat16)
    return q, kc, kb, torch.zeros(2, dtype=torch.int32)


def test_binding_checks_a_tree():
    plan, (q, kc, kb, lens) = shape_only_plan(), decode_inputs()
    out = torch.zeros(2, 4, 8, 64)
    with pytest.raises(ValueError, match="parents: 7"):
        plan.block_attn_tree(q, kc, kc, kb, kb, lens, torch.zeros(7, dtype=torch.int32), out=out)
    with pytest.raises(TypeError, match="parents"):
        plan.block_attn_tree(q, kc, kc, kb, kb, lens, torch.zeros(2, 4, dtype=torch.int64), out=out)
    with pytest.raises(ValueError, match="cuda:0"):
        plan.block_attn_tree(q, kc, kc, kb, kb, lens, torch.zeros(2, 4, dtype=torch.int32), out=out)
    with pytest.raises(ValueError, match="page_table"):
        plan.block_attn_tree_paged(q, kc, kc, torch.zeros(3, 1, dtype=torch.int32), kb, kb, lens,
                                   torch.zeros(2, 4, dtype=torch.int32), out=out)


def mx_cache(rows=2, heads=2, cap=32, dim=64, **kw):
    new = {"k": torch.zeros(rows, heads, cap, dim, dtype=torch.uint8),
           "k_scale": torch.zeros(rows, heads, cap, dim // 32, dtype=torch.uint8),
           "v": torch.zeros(rows, heads, cap, dim, dtype=torch.float8_e4m3fn),
           "v_scale": torch.zeros(rows, heads, cap, dim // 32, dtype=torch.uint8)}
    return ops.MxCache(**{**new, **kw})


def test_binding_checks_a_cache():
    mx_cache()
    with pytest.raises(ValueError, match="k: shape"):
        mx_cache(k=torch.zeros(4, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="k: shape"):
        mx_cache(dim=48)
    with pytest.raises(ValueError, match="v_scale"):
        mx_cache(v_scale=torch.zeros(3, dtype=torch.uint8))
    with pytest.raises(TypeError, match="k_scale"):
        mx_cache(k_scale=torch.zeros(2, 2, 32, 2))
    with pytest.raises(ValueError, match="page_table"):
        mx_cache(page_table=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="page_table"):
        mx_cache(page_table=torch.zeros(2, 1, dtype=torch.int64))


def test_binding_checks_rows_of_a_cache():
    plan, (q, _, kb, lens) = shape_only_plan(), decode_inputs()
    rows = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    for bad in (rows[:1], rows[:, :, :1], rows[..., :32], rows[0]):
        with pytest.raises(ValueError, match="k_new"):
            plan.kv_append_mx(bad, bad, mx_cache(), lens)
    with pytest.raises(ValueError, match="v_new"):
        plan.kv_append_mx(rows, rows[:, :2].contiguous(), mx_cache(), lens)
    with pytest.raises(ValueError, match="k_out"):
        plan.kv_read_mx(mx_cache(), lens, None, rows, rows)
    with pytest.raises(ValueError, match="starts"):
        out = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
        plan.kv_read_mx(mx_cache(), lens, torch.zeros(3, dtype=torch.int32), out, out)
    plan.device = -1          # the tensors' own "device": only the cache's shape is left to refuse
    with pytest.raises(ValueError, match="cache: shape"):
        plan.block_attn_mx(q, mx_cache(cap=16), kb, kb, lens, out=torch.zeros(2, 4, 8, 64))
    with pytest.raises(ValueError, match="cache: pages"):
        plan.block_attn_mx(q, mx_cache(page_table=torch.zeros(3, 1, dtype=torch.int32)), kb, kb, lens,
                           out=torch.zeros(2, 4, 8, 64))
