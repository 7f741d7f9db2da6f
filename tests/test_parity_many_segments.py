"""Few long units, each cut into dozens of segments: in the separate combine kernel and in the attention kernel's
tail, where up to four threads share an item."""
import numpy as np
import pytest
import torch

from oracle import visibility as vis
from tests.gpu_util import assert_parity, dev, f64, poison_beyond
from tests.test_parity import make_plan
from tests.test_parity_visibility import i32, poison_absent, tree_cases
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import make_decode

pytestmark = pytest.mark.gpu

KERNELS = [pytest.param((ops.KERNEL_TCGEN05, {}), id="tcgen05"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_FUSED_COMBINE": "1"}), id="fused"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_FUSED_COMBINE": "0"}), id="separate"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_TCGEN05_VARIANT": "2"}), id="transposed_pv"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_TCGEN05_VARIANT": "3"}), id="2sm"),
           pytest.param((ops.KERNEL_MMA_SYNC, {}), id="mma_sync")]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens", [[5000], [5000, 333], [5000] * 4, [4800, 5000, 1, 0]])
@pytest.mark.parametrize("S,g,D", [(16, 16, 128), (1, 16, 128), (5, 3, 64), (16, 8, 64), (85, 3, 64)])
def test_few_long_units(S, g, D, lens, tree, kernel):
    B, Hkv = len(lens), 2
    inp = make_decode(B, S, g * Hkv, Hkv, D, 5000, seed=101, ctx_lens=lens)
    par = None
    q, kb, vb = inp.q, inp.k_blk, inp.v_blk
    if tree:
        par = tree_cases(B, S, np.random.default_rng(102))
        q, kb, vb = poison_absent(inp, par)
    plan = make_plan(kernel, B, g * Hkv, Hkv, D, S, ctx_capacity=5000)
    x = [dev(t) for t in (q, poison_beyond(inp.k_ctx, lens), poison_beyond(inp.v_ctx, lens), kb, vb)]
    if tree:
        out, lse = plan.block_attn_tree(*x, i32(lens), i32(par), want_lse=True)
    else:
        out, lse = plan.block_attn(*x, i32(lens), want_lse=True)
    plan.check()
    ro, rl = vis.block_attn_visible(f64(inp.q), f64(inp.k_ctx), f64(inp.v_ctx), f64(inp.k_blk), f64(inp.v_blk), lens,
                                    parents=par)
    gone = np.isinf(rl)
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), gone)
    assert not out.cpu().numpy()[gone.transpose(0, 2, 1)].any()
    assert_parity(out, ro, "out")
    assert_parity(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse), np.where(gone, 0.0, rl), "lse")


@pytest.mark.parametrize("kernel", KERNELS[:3] + KERNELS[-1:])
@pytest.mark.parametrize("B,Hkv", [(4, 1), (40, 2), (64, 2)])
def test_short_lengths_in_a_large_capacity(B, Hkv, kernel):
    """Units of at most six tiles, which the capacity does not tell: cut where they are few, whole where they are
    many; then the same plan with one long sequence among them."""
    S, g, D, cap = 4, 4, 64, 2000
    rng = np.random.default_rng(103)
    plan = make_plan(kernel, B, g * Hkv, Hkv, D, S, ctx_capacity=cap)
    for longest in (300, 2000, 300):
        lens = [int(x) for x in rng.integers(0, 300, B)]
        lens[1] = longest
        inp = make_decode(B, S, g * Hkv, Hkv, D, cap, seed=104, ctx_lens=lens)
        x = [dev(t) for t in (inp.q, poison_beyond(inp.k_ctx, lens), poison_beyond(inp.v_ctx, lens), inp.k_blk, inp.v_blk)]
        out, lse = plan.block_attn(*x, i32(lens), want_lse=True)
        plan.check()
        ro, rl = vis.block_attn_visible(f64(inp.q), f64(inp.k_ctx), f64(inp.v_ctx), f64(inp.k_blk), f64(inp.v_blk), lens)
        assert_parity(out, ro, f"out, longest {longest}")
        assert_parity(lse, rl, f"lse, longest {longest}")
