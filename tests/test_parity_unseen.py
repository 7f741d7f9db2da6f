"""Context rows that no block sees hold NaN: none of a windowed block-causal call's results may show it, though
the partial tiles of the sinks and of the window are loaded in whole."""
import numpy as np
import pytest
import torch

from oracle import visibility as vis
from tests.gpu_util import BF16_NAN, assert_parity, dev, f64
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import bf16_bits, make_causal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bwd", ["tcgen05", "mma_sync"])
@pytest.mark.parametrize("window,sinks", [(5, 3), (9, 0), (3, 17)])
@pytest.mark.parametrize("S,Hq,Hkv,D", [(16, 8, 2, 128), (16, 32, 2, 128), (16, 16, 2, 64), (21, 6, 2, 64)])
def test_block_causal_with_unseen_rows_of_nan(S, Hq, Hkv, D, window, sinks, bwd, monkeypatch):
    B, N = 2, 24 * S
    inp = make_causal(B, N, S, Hq, Hkv, D, seed=71)
    seen = np.zeros(N, dtype=bool)
    for b in range(N // S):
        seen[:S * b] |= vis.visible_context(S * b, window, sinks)
    assert not seen.all()
    kc, vc = inp.k_ctx.copy(), inp.v_ctx.copy()
    kc[:, :, ~seen] = BF16_NAN
    vc[:, :, ~seen] = BF16_NAN
    dout = bf16_bits(np.random.default_rng(72).standard_normal((B, N, Hq, D)).astype(np.float32))
    monkeypatch.setenv("TT_BWD_KERNEL", bwd)
    plan = ops.Plan(B, Hq, Hkv, D, S, seq_len=N, window=window, sinks=sinks)
    x = [dev(t) for t in (inp.q, kc, vc, inp.k_blk, inp.v_blk)]
    out, lse = plan.block_attn_block_causal(*x, want_lse=True)
    for _ in range(20):   # the order of a clear and its reader varies
        grads = plan.block_causal_backward(*x, out, lse, dev(dout))
        assert all(bool(torch.isfinite(g).all()) for g in grads)
    plan.check()
    y = [f64(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)]
    ro, rl = vis.block_causal_window(*y, S, window, sinks)
    assert_parity(out, ro, "out")
    assert_parity(lse, rl, "lse")
    for name, got, ref in zip(("dq", "dk_blk", "dv_blk"), grads,
                              vis.block_causal_window_backward(*y, f64(dout), S, window, sinks)):
        assert_parity(got, ref, name)
