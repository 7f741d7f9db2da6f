"""A NaN in the quantised cache shows: e4m3's NaN makes NaN of the rows that see it and of no others, on every
kernel and whichever range of a cut unit met it."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from oracle import visibility as vis
from tests.gpu_util import assert_parity, dev, f64
from tests.test_parity import make_plan
from tests.test_parity_mx import device_cache, paged_cache
from tests.test_parity_visibility import i32
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import make_decode

pytestmark = pytest.mark.gpu

TC = ops.KERNEL_TCGEN05
KERNELS = [pytest.param((TC, {}), id="tcgen05"), pytest.param((TC, {"TT_FUSED_COMBINE": "1"}), id="fused"),
           pytest.param((ops.KERNEL_MMA_SYNC, {}), id="mma_sync")]
#            B, S, Hq, Hkv, D, Lcap, lens
SHAPES = {"two_m_tiles": (2, 16, 32, 2, 128, 700, [700, 300]), "one_m_tile": (2, 4, 16, 2, 64, 700, [699, 64])}


def case(shape, window=0, sinks=0):
    B, S, Hq, Hkv, D, cap, lens = SHAPES[shape]
    inp = make_decode(B, S, Hq, Hkv, D, cap, seed=51, ctx_lens=lens)
    q = [omx.quantise(f64(x)) for x in (inp.k_ctx, inp.v_ctx)]
    host = [*q[0], *q[1]]
    ref = vis.block_attn_visible(f64(inp.q), omx.values(*host[:2]), omx.values(*host[2:]), f64(inp.k_blk),
                                 f64(inp.v_blk), lens, window, sinks)
    return inp, host, ref


def run(kernel, shape, inp, host, num_ctas, page=0, **kw):
    B, S, Hq, Hkv, D, cap, lens = SHAPES[shape]
    plan = make_plan(kernel, B, Hq, Hkv, D, S, ctx_capacity=cap, num_ctas=num_ctas, **kw)
    cache = paged_cache(host, page, 52, lens) if page else device_cache(host)
    out, lse = plan.block_attn_mx(dev(inp.q), cache, dev(inp.k_blk), dev(inp.v_blk), i32(lens), want_lse=True)
    plan.check()
    return out, lse


def check(out, lse, ref, gone):
    """gone [B, Hq, S]: rows that have to be NaN, all others as in ref."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = np.moveaxis(gone, 1, 2)
    assert np.isnan(out[rows]).all()
    assert_parity(torch.from_numpy(out[~rows]), ref[0][~rows], "out")
    assert np.isnan(lse[gone]).all()
    assert_parity(torch.from_numpy(lse[~gone]), ref[1][~gone], "lse")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("num_ctas,page", [(0, 0), (5, 0), (0, 16)])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("where,code", [(0, 0x7F), (63, 0xFF), (64, 0x7F), (450, 0x7F), ("last", 0xFF)])
def test_a_nan_key_shows(where, code, shape, num_ctas, page, kernel):
    B, S, Hq, Hkv, D, cap, lens = SHAPES[shape]
    inp, host, ref = case(shape)
    host[0][0, 1, lens[0] - 1 if where == "last" else where, D - 1] = code
    gone = np.zeros((B, Hq, S), dtype=bool)
    gone[0, Hq // Hkv:] = True
    check(*run(kernel, shape, inp, host, num_ctas, page), ref, gone)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("num_ctas,page", [(0, 0), (5, 16)])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("scale", [0, 127, 200])
@pytest.mark.parametrize("where", [0, 130, "last"])
def test_a_nan_value_shows_in_its_column(where, scale, shape, num_ctas, page, kernel):
    """The value's scale is of no account: the column of the output is NaN, the others and lse are not."""
    B, S, Hq, Hkv, D, cap, lens = SHAPES[shape]
    inp, host, _ = case(shape)
    pos, col = (lens[1] - 1 if where == "last" else min(where, lens[1] - 1)), 33
    host[2][1, 0, pos, 32:64] = 0        # the rest of its scale block: zeros, whatever the scale
    host[3][1, 0, pos, 1] = scale
    ref = vis.block_attn_visible(f64(inp.q), omx.values(*host[:2]), omx.values(*host[2:]), f64(inp.k_blk),
                                 f64(inp.v_blk), lens)
    host[2][1, 0, pos, col] = 0xFF
    out, lse = run(kernel, shape, inp, host, num_ctas, page)
    out = out.double().cpu()
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[1, :, :Hq // Hkv, col] = True
    assert torch.isnan(out[hit]).all()
    assert_parity(out[~hit], ref[0][~hit.numpy()], "out")
    assert_parity(lse, ref[1], "lse")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_a_nan_outside_the_window_does_not(shape, page, kernel):
    B, S, Hq, Hkv, D, cap, lens = SHAPES[shape]
    inp, host, ref = case(shape, 70, 20)
    for n, L in enumerate(lens):
        for a in (host[0], host[2]):
            a[n, :, 20:max(20, L - 70)] = 0x7F
    check(*run(kernel, shape, inp, host, 0, page, window=70, sinks=20), ref, np.zeros((B, Hq, S), dtype=bool))
