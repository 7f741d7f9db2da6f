"""Units of at most 128 rows, whose tiles two softmax warpgroups take in turn: many tiles and several units in one
CTA, so that every slot of the rings is used again and again by either of them."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from oracle import visibility as vis
from tests.gpu_util import assert_parity, dev, f64, poison_beyond
from tests.test_parity_mx import device_cache, paged_cache
from tests.test_parity_visibility import i32, tree_cases
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import make_decode

pytestmark = pytest.mark.gpu

CAP, LENS = 8192, [8192, 5001]


def case(S, g, D):
    inp = make_decode(2, S, 2 * g, 2, D, CAP, seed=91, ctx_lens=LENS)
    q = [omx.quantise(f64(x)) for x in (inp.k_ctx, inp.v_ctx)]
    return inp, (*q[0], *q[1])


def reference(inp, k, v, parents=None):
    ro, rl = vis.block_attn_visible(f64(inp.q), k, v, f64(inp.k_blk), f64(inp.v_blk), LENS, parents=parents)
    return ro, np.where(np.isinf(rl), 0.0, rl)


def check(calls, ref):
    first = None
    for _ in range(4):   # the interleaving varies, the result must not
        out, lse = calls()
        lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
        if first is None:
            first = out.clone(), lse.clone()
            assert_parity(out, ref[0], "out")
            assert_parity(lse, ref[1], "lse")
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("num_ctas", [1, 3, 5])
@pytest.mark.parametrize("page", [0, 16, 32])
@pytest.mark.parametrize("S,g,D", [(1, 16, 64), (1, 16, 128), (8, 16, 128), (5, 3, 64)])
def test_quantised_cache(S, g, D, page, num_ctas):
    inp, host = case(S, g, D)
    plan = ops.Plan(2, 2 * g, 2, D, S, ctx_capacity=CAP, num_ctas=num_ctas)
    cache = paged_cache(host, page, 92, LENS) if page else device_cache(host)
    x = dev(inp.q), dev(inp.k_blk), dev(inp.v_blk)
    check(lambda: plan.block_attn_mx(x[0], cache, x[1], x[2], i32(LENS), want_lse=True),
          reference(inp, omx.values(*host[:2]), omx.values(*host[2:])))
    plan.check()


@pytest.mark.parametrize("num_ctas", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_quantised_cache_with_a_tree(D, num_ctas):
    S, g = 70, 1      # two block tiles a unit
    inp, host = case(S, g, D)
    par = tree_cases(2, S, np.random.default_rng(93))
    plan = ops.Plan(2, 2 * g, 2, D, S, ctx_capacity=CAP, num_ctas=num_ctas)
    cache = device_cache(host)
    x = dev(inp.q), dev(inp.k_blk), dev(inp.v_blk)
    check(lambda: plan.block_attn_mx(x[0], cache, x[1], x[2], i32(LENS), parents=i32(par), want_lse=True),
          reference(inp, omx.values(*host[:2]), omx.values(*host[2:]), par))
    plan.check()


@pytest.mark.parametrize("num_ctas", [1, 3, 5])
@pytest.mark.parametrize("S,g,D", [(1, 16, 64), (1, 16, 128), (8, 16, 128), (5, 3, 64)])
def test_bf16_cache(S, g, D, num_ctas):
    inp, _ = case(S, g, D)
    plan = ops.Plan(2, 2 * g, 2, D, S, ctx_capacity=CAP, num_ctas=num_ctas)
    x = [dev(t) for t in (inp.q, poison_beyond(inp.k_ctx, LENS), poison_beyond(inp.v_ctx, LENS), inp.k_blk, inp.v_blk)]
    check(lambda: plan.block_attn(*x, i32(LENS), want_lse=True), reference(inp, f64(inp.k_ctx), f64(inp.v_ctx)))
    plan.check()
