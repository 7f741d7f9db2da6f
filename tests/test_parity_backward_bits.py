"""The block's gradients take the weights in 32 bits."""
import numpy as np
import pytest
import torch

from tests.gpu_util import dev, f64
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import bf16_bits, make_causal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_a_single_row_gives_dv_to_32_bits(D):
    """One query row a block: dv = p dO is one product, p = exp(scale q.k - lse) with the lse that the call is
    given.  The scores are below 2^-2, so p's argument is lse in log2 units, below 2^3, rounded twice
    (2^-21 each), times ln 2, plus 2 ulp of the exponential (2^-22) and the product's rounding (2^-23):
    1.2e-6, below 2^-19.  Weights held in two bf16 parts are off by up to 2^-18."""
    B, N, H = 2, 200, 4
    rng = np.random.default_rng(81)
    inp = make_causal(B, N, 1, H, H, D, seed=82)
    q = bf16_bits(f64(inp.q).astype(np.float32) * 2.0 ** -6)
    dout = bf16_bits(rng.standard_normal((B, N, H, D)).astype(np.float32))
    plan = ops.Plan(B, H, H, D, 1, seq_len=N)
    x = [dev(t) for t in (q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)]
    out, lse = plan.block_attn_block_causal(*x, want_lse=True)
    _, _, dv = plan.block_causal_backward(*x, out, lse, dev(dout))
    plan.check()
    s = np.einsum("bnhd,bnhd->bhn", f64(q), f64(inp.k_blk)) / np.sqrt(D)
    assert np.abs(s).max() < 0.25 and lse.max() < 5.5
    p = np.exp(s - lse.double().cpu().numpy()).transpose(0, 2, 1)[..., None]
    ref = p * f64(dout)
    off = np.abs(dv.double().cpu().numpy() - ref) / np.abs(ref)
    assert off.max() <= 2.0 ** -19
