"""Sizes at the edges of what the calls accept."""
import pytest
import torch

from oracle import visibility as vis
from tests.gpu_util import assert_parity, dev, f64
from tests.test_parity_visibility import i32
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import make_decode, make_paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", [ops.KERNEL_TCGEN05, ops.KERNEL_MMA_SYNC])
@pytest.mark.parametrize("window", [0, 1500])
def test_a_page_table_of_the_widest_capacity(window, kernel):
    """2^31 - 16 positions a sequence (a table row of 2^27 - 1 entries): the tile count of the capacity must not
    pass 32 bits, or long units would be cut with no combine to follow."""
    B, S, Hq, Hkv, D, L = 1, 4, 8, 1, 64, 3000
    inp = make_decode(B, S, Hq, Hkv, D, L, seed=61, ctx_lens=[L])
    pages = make_paged(inp, 16, seed=62)
    table = torch.zeros(B, (1 << 27) - 1, dtype=torch.int32, device="cuda")
    small = torch.from_numpy(pages.page_table).cuda()
    table[:, :small.shape[1]] = small
    plan = ops.Plan(B, Hq, Hkv, D, S, window=window, kernel=kernel)
    out, lse = plan.block_attn_paged(dev(inp.q), dev(pages.k_pages), dev(pages.v_pages), table, dev(inp.k_blk),
                                     dev(inp.v_blk), i32([L]), out=torch.full((B, S, Hq, D), 7.0, device="cuda"),
                                     want_lse=True)
    plan.check()
    ro, rl = vis.block_attn_visible(f64(inp.q), f64(inp.k_ctx), f64(inp.v_ctx), f64(inp.k_blk), f64(inp.v_blk), [L],
                                    window, 0)
    assert_parity(out, ro, "out")
    assert_parity(lse, rl, "lse")


@pytest.mark.parametrize("B,Hkv,status", [(32, 1, ops.TT_OK), (33, 2, ops.TT_ERR_UNSUPPORTED),
                                          (64, 1, ops.TT_ERR_UNSUPPORTED)])
def test_tables_whose_capacities_pass_the_tile_count_are_refused(B, Hkv, status):
    """Sequences that share pages may have more positions together than a pool has rows; their tiles are counted
    in 32 bits.  (No table entry is read here: every length is 0.)"""
    S, D = 4, 64
    x = [torch.zeros(B, S, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hkv)]
    pool = torch.zeros(1, Hkv, 16, D, dtype=torch.bfloat16, device="cuda")
    table, lens = i32([[0]] * B), i32([0] * B)
    out = torch.empty(B, S, Hkv, D, device="cuda")
    plan = ops.Plan(B, Hkv, Hkv, D, S)
    p = ops._ptr
    got = ops.lib().tt_block_attn_paged(plan._h, p(x[0]), p(pool), p(pool), p(table), 1, 16, (1 << 27) - 1, p(x[1]),
                                        p(x[2]), p(lens), p(out), None, ops._stream(plan))
    assert got == status
    plan.check()


def test_a_quantised_cache_of_many_sequences():
    B, D = 70001, 64
    cache = ops.MxCache.empty(B, 1, 2, D)
    plan = ops.Plan(B, 1, 1, D, 1, ctx_capacity=2)
    rows = torch.arange(B, device="cuda").remainder(449).sub(224).to(torch.bfloat16)
    rows = rows[:, None, None, None].expand(B, 1, 1, D).contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for step in (1, 2):
        plan.kv_append_mx(rows * step, -rows, cache, lens)
        assert bool((lens == step).all())
    k, v = (torch.full((B, 1, 2, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    plan.kv_read_mx(cache, lens, None, k, v)
    plan.check()
    # equal elements: the scale is a power of two, so each reads as e4m3 of its mantissa, within 2^-4
    want = rows[:, :, 0].float()
    for got, ref in ((k[:, :, 0], want), (k[:, :, 1], 2 * want), (v[:, :, 0], -want), (v[:, :, 1], -want)):
        assert bool(((got.float() - ref).abs() <= 2.0 ** -4 * ref.abs()).all())
