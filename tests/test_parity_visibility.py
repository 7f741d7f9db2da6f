"""GPU parity of windowed layers (sliding window and sinks) and of drafted trees against the float64
oracle, on the default tcgen05 kernel and the mma.sync kernel.

Tolerance: the framework's bar (max-abs <= 1e-2, relative L2 <= 5e-3).  What it has to hold here:
the weights are rounded to bf16 (relative error at most 2^-8, the same rounded weights in numerator
and denominator), so |out - ref| <= 2^-8 sum_k w_k |v_k - out| per element; with v ~ N(0, 1) the mean
absolute deviation is about 0.8, hence about 3e-3, and one weight in eight adds 7.5e-5.

Everything that must not be read or must not matter is NaN: context rows that are not visible, rows
of a window's first page that lie before the window, pages outside the window (their table entries are
-1), and q, k and v of absent tree rows."""
import numpy as np
import pytest
import torch

from oracle import visibility as vis
from tests.gpu_util import BF16_NAN, assert_parity, dev, f64
from tests.test_parity import make_plan
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import bf16_bits, make_causal, make_decode, make_paged

pytestmark = pytest.mark.gpu

KERNELS = [pytest.param((ops.KERNEL_TCGEN05, {}), id="tcgen05"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_FUSED_COMBINE": "1"}), id="tcgen05_fused"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_FUSED_COMBINE": "0"}), id="tcgen05_separate"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_TCGEN05_KEY_TILE": "128"}), id="tcgen05_k128"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_TCGEN05_VARIANT": "3"}), id="tcgen05_2sm"),
           pytest.param((ops.KERNEL_MMA_SYNC, {}), id="mma_sync")]
SOME = [KERNELS[0], KERNELS[1], KERNELS[5]]


def poison_hidden(bits, lens, window, sinks):
    """Copy of a [B, Hkv, Lcap, D] cache with every row that no block sees set to NaN."""
    k = np.full_like(bits, BF16_NAN)
    for n, L in enumerate(lens):
        c = np.flatnonzero(vis.visible_context(int(L), window, sinks))
        k[n, :, c] = bits[n, :, c]
    return k


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def check_decode(inp, out, lse, window=0, sinks=0, parents=None, what=""):
    ro, rl = vis.block_attn_visible(f64(inp.q), f64(inp.k_ctx), f64(inp.v_ctx), f64(inp.k_blk), f64(inp.v_blk),
                                    inp.ctx_lens, window, sinks, parents)
    if parents is not None:
        gone = np.isinf(rl)
        assert np.array_equal(np.isneginf(lse.cpu().numpy()), gone), f"{what}: rows that see nothing"
        rl = np.where(gone, 0.0, rl)
        lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
        rows = gone.transpose(0, 2, 1)          # [B, S, Hq]
        assert not out.float().cpu().numpy()[rows].any(), f"{what}: an absent row's output is 0"
    assert_parity(out, ro, f"{what} out")
    assert_parity(lse, rl, f"{what} lse")


# B, S, Hq, Hkv, D, Lcap, lens
SHAPES = {
    "S16-g16": (5, 16, 32, 2, 128, 700, [700, 0, 1, 300, 129]),
    "S1-g16": (4, 1, 16, 1, 128, 513, [513, 0, 1, 255]),
    "S5-g3-d64": (3, 5, 6, 2, 64, 200, [200, 64, 17]),
    "S64-g4": (2, 64, 8, 2, 128, 400, [400, 193]),
    "S200-g1-d64": (2, 200, 2, 2, 64, 300, [300, 65]),
}
# window, sinks: one key; no sinks; sinks over a tile; runs that touch; a window beyond every context
WINDOWS = [(1, 0), (64, 0), (100, 4), (130, 70), (63, 1), (300, 400), (5000, 3)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_window_decode(shape, window, sinks, kernel):
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES[shape]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=50, ctx_lens=lens)
    plan = make_plan(kernel, B, Hq, Hkv, D, S, ctx_capacity=Lcap, window=window, sinks=sinks)
    kc, vc = (poison_hidden(x, lens, window, sinks) for x in (inp.k_ctx, inp.v_ctx))
    out, lse = plan.block_attn(dev(inp.q), dev(kc), dev(vc), dev(inp.k_blk), dev(inp.v_blk), i32(lens), want_lse=True)
    plan.check()
    check_decode(inp, out, lse, window, sinks, what=f"{shape} W={window} s={sinks}")


def windowed_pages(inp, page_size, window, sinks, seed):
    """make_paged with NaN in every row that is not visible and -1 for pages without a visible row."""
    lens = inp.ctx_lens
    hidden = type(inp)(**{**inp.__dict__, "k_ctx": poison_hidden(inp.k_ctx, lens, window, sinks),
                          "v_ctx": poison_hidden(inp.v_ctx, lens, window, sinks)})
    pc = make_paged(hidden, page_size, seed=seed)
    for n, L in enumerate(lens):
        seen = set(np.flatnonzero(vis.visible_context(int(L), window, sinks)) // page_size)
        for i in range(pc.page_table.shape[1]):
            if i not in seen:
                pc.page_table[n, i] = -1
    return pc


@pytest.mark.parametrize("kernel", SOME)
@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (130, 70), (300, 400)])
@pytest.mark.parametrize("shape", ["S16-g16", "S1-g16", "S5-g3-d64"])
def test_window_paged(shape, window, sinks, page_size, kernel):
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES[shape]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=51, ctx_lens=lens)
    pc = windowed_pages(inp, page_size, window, sinks, seed=page_size)
    plan = make_plan(kernel, B, Hq, Hkv, D, S, window=window, sinks=sinks)
    out, lse = plan.block_attn_paged(dev(inp.q), dev(pc.k_pages), dev(pc.v_pages), i32(pc.page_table), dev(inp.k_blk),
                                     dev(inp.v_blk), i32(lens), want_lse=True)
    plan.check()
    check_decode(inp, out, lse, window, sinks, what=f"{shape} P={page_size} W={window} s={sinks}")


@pytest.mark.parametrize("num_ctas", [1, 3, 37, 148, 300])
def test_window_split_invariance(num_ctas):
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES["S16-g16"]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=52, ctx_lens=lens)
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, window=200, sinks=9, num_ctas=num_ctas)
    out, lse = plan.block_attn(dev(inp.q), dev(inp.k_ctx), dev(inp.v_ctx), dev(inp.k_blk), dev(inp.v_blk), i32(lens),
                               want_lse=True)
    plan.check()
    check_decode(inp, out, lse, 200, 9, what=f"C={num_ctas}")


def test_window_over_everything_equals_the_plain_plan_bit_for_bit():
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES["S16-g16"]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=53, ctx_lens=lens)
    x = [dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)] + [i32(lens)]
    got = [ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, num_ctas=100, **kw).block_attn(*x, want_lse=True)
           for kw in ({}, {"window": Lcap}, {"window": 600, "sinks": 200})]
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_window_host_buffers_equal_the_device_call():
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES["S5-g3-d64"]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=54, ctx_lens=lens)
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, window=50, sinks=2, host_io=True)
    x = [dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)] + [i32(lens)]
    want = plan.block_attn(*x)
    out = torch.empty(want.shape, pin_memory=True)
    plan.block_attn_host(*[t.cpu().pin_memory() for t in x], out)
    plan.check()
    assert torch.equal(out, want.cpu())


CAUSAL = [  # B, N, S, Hq, Hkv, D, window, sinks
    (1, 320, 16, 32, 2, 128, 70, 5), (2, 192, 4, 8, 2, 64, 33, 0), (1, 300, 5, 6, 2, 128, 64, 130),
    (1, 256, 8, 16, 1, 128, 1, 1), (1, 128, 1, 16, 1, 64, 20, 2), (1, 512, 64, 8, 2, 128, 100, 3),
]


@pytest.mark.parametrize("bwd", ["tcgen05", "mma_sync"])
@pytest.mark.parametrize("kernel", [KERNELS[0], KERNELS[3], KERNELS[5]])
@pytest.mark.parametrize("shape", CAUSAL)
def test_window_block_causal_and_backward(shape, kernel, bwd, monkeypatch):
    """Forward and gradients; the backward's bar and its reasons are those of the unwindowed one."""
    B, N, S, Hq, Hkv, D, window, sinks = shape
    inp = make_causal(B, N, S, Hq, Hkv, D, seed=55)
    dout = bf16_bits(np.random.default_rng(56).standard_normal((B, N, Hq, D)).astype(np.float32))
    plan = make_plan(kernel, B, Hq, Hkv, D, S, seq_len=N, window=window, sinks=sinks)
    x = [dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)]
    out, lse = plan.block_attn_block_causal(*x, want_lse=True)
    monkeypatch.setenv("TT_BWD_KERNEL", bwd)
    grads = plan.block_causal_backward(*x, out, lse, dev(dout))
    plan.check()
    y = [f64(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)]
    ro, rl = vis.block_causal_window(*y, S, window, sinks)
    assert_parity(out, ro, "out")
    assert_parity(lse, rl, "lse")
    for name, got, ref in zip(("dq", "dk_blk", "dv_blk"), grads,
                              vis.block_causal_window_backward(*y, f64(dout), S, window, sinks)):
        assert_parity(got, ref, name)


# ----------------------------------------------------------------------- trees --
def random_parents(rng, B, S):
    par = np.array([[rng.integers(-1, t) if t else -1 for t in range(S)] for _ in range(B)], dtype=np.int32)
    return par


def tree_cases(B, S, rng):
    """Random trees, a chain, a star, some rows absent, and one sequence without any row."""
    par = random_parents(rng, B, S)
    par[0] = np.arange(S) - 1
    if B > 1:
        par[1] = -1
    if B > 2:
        par[2, S // 2] = -2
    if B > 3:
        par[3] = -2
    if B > 4:
        par[4, (S + 1) // 2:] = -2
    return par


def poison_absent(inp, parents):
    q, k, v = inp.q.copy(), inp.k_blk.copy(), inp.v_blk.copy()
    for n in range(len(parents)):
        gone = ~vis.tree_visibility(parents[n])[1]
        for a in (q, k, v):
            a[n, gone] = BF16_NAN
    return q, k, v


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_tree_decode(shape, kernel):
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES[shape]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=60, ctx_lens=lens)
    par = tree_cases(B, S, np.random.default_rng(61))
    q, kb, vb = poison_absent(inp, par)
    plan = make_plan(kernel, B, Hq, Hkv, D, S, ctx_capacity=Lcap)
    kc, vc = (poison_hidden(x, lens, 0, 0) for x in (inp.k_ctx, inp.v_ctx))
    out, lse = plan.block_attn_tree(dev(q), dev(kc), dev(vc), dev(kb), dev(vb), i32(lens), i32(par), want_lse=True)
    plan.check()
    check_decode(inp, out, lse, parents=par, what=shape)


@pytest.mark.parametrize("kernel", SOME)
@pytest.mark.parametrize("page_size", [16, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
@pytest.mark.parametrize("shape", ["S16-g16", "S5-g3-d64", "S64-g4", "S200-g1-d64"])
def test_tree_paged_with_and_without_a_window(shape, window, sinks, page_size, kernel):
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES[shape]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=62, ctx_lens=lens)
    par = tree_cases(B, S, np.random.default_rng(63))
    q, kb, vb = poison_absent(inp, par)
    pc = windowed_pages(inp, page_size, window, sinks, seed=page_size)
    plan = make_plan(kernel, B, Hq, Hkv, D, S, window=window, sinks=sinks, out_bf16=True)
    out, lse = plan.block_attn_tree_paged(dev(q), dev(pc.k_pages), dev(pc.v_pages), i32(pc.page_table), dev(kb),
                                          dev(vb), i32(lens), i32(par), want_lse=True)
    plan.check()
    assert out.dtype == torch.bfloat16
    # a bf16 output is off by at most 2^-8 of its value more: |out| <= 4 here, 1.6e-2 in all
    ro, rl = vis.block_attn_visible(f64(inp.q), f64(inp.k_ctx), f64(inp.v_ctx), f64(inp.k_blk),
                                    f64(inp.v_blk), inp.ctx_lens, window, sinks, par)
    assert_parity(out, ro, "out", max_abs=1e-2 + 2.0 ** -8 * float(np.abs(ro).max()), rel_l2=5e-3 + 2.0 ** -8)
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), np.isneginf(rl))


@pytest.mark.parametrize("num_ctas", [1, 5, 148, 300])
@pytest.mark.parametrize("shape", ["S16-g16", "S200-g1-d64"])
def test_tree_split_invariance(shape, num_ctas):
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES[shape]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=64, ctx_lens=lens)
    par = tree_cases(B, S, np.random.default_rng(65))
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, num_ctas=num_ctas)
    out, lse = plan.block_attn_tree(dev(inp.q), dev(inp.k_ctx), dev(inp.v_ctx), dev(inp.k_blk), dev(inp.v_blk),
                                    i32(lens), i32(par), want_lse=True)
    plan.check()
    check_decode(inp, out, lse, parents=par, what=f"C={num_ctas}")


def test_tree_of_one_token_equals_plain_decode():
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES["S1-g16"]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=66, ctx_lens=lens)
    x = [dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)] + [i32(lens)]
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap)
    want = plan.block_attn(*x)
    got = plan.block_attn_tree(*x, i32(np.full((B, 1), -1)))
    plan.check()
    # the masked tile takes every weight with the hardware exp2, the plain one some by polynomial
    assert float((got - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max())


@pytest.mark.parametrize("kernel", SOME)
@pytest.mark.parametrize("bad", [(0, 2, 2), (1, 0, 5), (1, 3, -3), (0, 1, 2 ** 30)])
def test_tree_bad_parent_is_flagged_and_its_row_absent(bad, kernel):
    B, S, Hq, Hkv, D, Lcap, lens = 2, 6, 8, 2, 64, 100, [100, 30]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=67, ctx_lens=lens)
    par = random_parents(np.random.default_rng(68), B, S)
    n, t, value = bad
    par[n, t] = value
    plan = make_plan(kernel, B, Hq, Hkv, D, S, ctx_capacity=Lcap)
    out, lse = plan.block_attn_tree(dev(inp.q), dev(inp.k_ctx), dev(inp.v_ctx), dev(inp.k_blk), dev(inp.v_blk),
                                    i32(lens), i32(par), want_lse=True)
    assert plan.check_status() == ops.TT_ERR_DEVICE_ARG
    par[n, t] = -2
    check_decode(inp, out, lse, parents=par, what="bad parent")


def test_window_and_tree_in_graphs_and_on_another_stream():
    """One captured graph of a windowed, a tree and a plain call, replayed with new lengths; the same
    calls on a side stream."""
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES["S16-g16"]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=69, ctx_lens=lens)
    par = tree_cases(B, S, np.random.default_rng(70))
    x = [dev(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)]
    lens_d, par_d = i32(lens), i32(par)
    pw = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, window=100, sinks=4)
    pt = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap)
    outs = [torch.empty((B, S, Hq, D), device="cuda") for _ in range(3)]

    def calls():
        pw.block_attn(*x, lens_d, out=outs[0])
        pt.block_attn_tree(*x, lens_d, par_d, out=outs[1])
        pt.block_attn(*x, lens_d, out=outs[2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
        for new in (lens, [0, 700, 64, 65, 333]):
            lens_d.copy_(i32(new))
            for o in outs:
                o.fill_(7.0)
            graph.replay()
            side.synchronize()
            inp.ctx_lens = np.asarray(new, dtype=np.int32)
            y = [f64(t) for t in (inp.q, inp.k_ctx, inp.v_ctx, inp.k_blk, inp.v_blk)]
            for o, kw in zip(outs, (dict(window=100, sinks=4), dict(parents=par), {})):
                assert_parity(o, vis.block_attn_visible(*y, new, **kw)[0], str(kw.keys()))
    pw.check()
    pt.check()
