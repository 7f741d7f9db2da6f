"""GPU parity where a decode call keeps whole units (contexts of at most a few tiles: one launch, nothing
combined), around that limit, with more units than SMs, and into outputs whose alignment is the least that
is allowed.  Tolerance: the framework's bar, as tests/test_parity_visibility.py derives it."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from oracle import visibility as vis
from tests.gpu_util import assert_parity, dev, f64
from tests.test_parity_mx import device_cache
from tests.test_parity_visibility import check_decode, i32, poison_hidden, tree_cases
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import bf16_bits, make_causal, make_decode

pytestmark = pytest.mark.gpu

# B, S, Hq, Hkv, D, Lcap, lens: below the limit, across it (capacity above, lengths below and above), a
# batch of many units, one unit
SHORT = [(3, 16, 32, 2, 128, 300, [300, 0, 129]), (3, 16, 32, 2, 128, 700, [300, 0, 129]),
         (3, 5, 6, 2, 64, 700, [320, 321, 7]), (40, 3, 8, 4, 64, 200, list(range(0, 200, 5))),
         (1, 1, 16, 1, 128, 64, [64]), (2, 256, 1, 1, 128, 100, [100, 1])]


@pytest.mark.parametrize("form", ["plain", "window", "tree", "mx"])
@pytest.mark.parametrize("case", range(len(SHORT)))
def test_short_contexts(case, form):
    B, S, Hq, Hkv, D, Lcap, lens = SHORT[case]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=300 + case, ctx_lens=lens)
    kw = dict(window=90, sinks=5) if form == "window" else {}
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, **kw)
    par = tree_cases(B, S, np.random.default_rng(case)) if form == "tree" else None
    x = dev(inp.q), dev(inp.k_blk), dev(inp.v_blk)
    if form == "mx":
        q = [omx.quantise(f64(t)) for t in (inp.k_ctx, inp.v_ctx)]
        inp.k_ctx, inp.v_ctx = (bf16_bits(omx.values(*a).astype(np.float32)) for a in q)   # exact in bf16
        out, lse = plan.block_attn_mx(x[0], device_cache((*q[0], *q[1])), x[1], x[2], i32(lens), want_lse=True)
    else:
        kc, vc = (dev(poison_hidden(t, lens, kw.get("window", 0), kw.get("sinks", 0))) for t in (inp.k_ctx, inp.v_ctx))
        a = x[0], kc, vc, x[1], x[2], i32(lens)
        out, lse = plan.block_attn_tree(*a, i32(par), want_lse=True) if par is not None else \
            plan.block_attn(*a, want_lse=True)
    plan.check()
    check_decode(inp, out, lse, parents=par, what=f"{form} {case}", **kw)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("Lcap", [100, 900])
def test_outputs_of_the_least_alignment(Lcap, bf16):
    """An output 16 bytes into a 32-byte line equals the one at its start, bit for bit."""
    B, S, Hq, Hkv, D = 2, 16, 32, 2, 128
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=320)
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, out_bf16=bf16)
    a = [dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)] + [i32(inp.ctx_lens)]
    want = plan.block_attn(*a)
    n, off = want.numel(), 16 // want.element_size()
    buf = torch.full((n + 2 * off,), 7.0, dtype=want.dtype, device="cuda")
    plan.block_attn(*a, out=buf[off:off + n].view(want.shape))
    plan.check()
    assert torch.equal(buf[off:off + n].view(want.shape), want)
    assert (buf[:off] == 7).all() and (buf[off + n:] == 7).all()


def test_gradients_of_the_least_alignment():
    B, N, S, Hq, Hkv, D = 1, 160, 8, 8, 2, 128
    inp = make_causal(B, N, S, Hq, Hkv, D, seed=321)
    dout = dev(bf16_bits(np.random.default_rng(322).standard_normal((B, N, Hq, D)).astype(np.float32)))
    plan = ops.Plan(B, Hq, Hkv, D, S, seq_len=N, window=40, sinks=2)
    a = [dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)]
    out, lse = plan.block_attn_block_causal(*a, want_lse=True)
    want = plan.block_causal_backward(*a, out, lse, dout)
    got = []
    for w in want:   # filled with NaN: what is not written shows
        buf = torch.full((w.numel() + 4,), float("nan"), device="cuda")
        got.append(buf[4:].view(w.shape))
    plan.block_causal_backward(*a, out, lse, dout, *got)
    plan.check()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_short_blocks_of_sequences():
    """Block-causal calls that keep whole units, with and without a window, against the oracle."""
    for N, S, window, sinks in ((96, 16, 0, 0), (320, 16, 64, 3), (40, 5, 7, 0)):
        B, Hq, Hkv, D = 1, 8, 2, 128
        inp = make_causal(B, N, S, Hq, Hkv, D, seed=330 + N)
        plan = ops.Plan(B, Hq, Hkv, D, S, seq_len=N, window=window, sinks=sinks)
        out, lse = plan.block_attn_block_causal(*[dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)],
                                                want_lse=True)
        plan.check()
        ro, rl = vis.block_causal_window(*[f64(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)], S,
                                         window, sinks)
        assert_parity(out, ro, f"N={N} out")
        assert_parity(lse, rl, f"N={N} lse")
