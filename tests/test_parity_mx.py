"""GPU checks of the microscaled context cache: the write bit for bit against the oracle, the read-back
exactly, attention over the cache against the float64 oracle on the values the cache stands for.

Attention's tolerance is the framework's bar; the cache adds nothing to it, since its values are exact
bf16 operands."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from oracle import visibility as vis
from tests.gpu_util import assert_parity, dev, f64
from tests.test_parity import make_plan
from tests.test_parity_visibility import SHAPES, i32, poison_absent, tree_cases
from two_tower_block_b200 import ops
from two_tower_block_b200.workloads import bf16_bits, make_decode

pytestmark = pytest.mark.gpu

KERNELS = [pytest.param((ops.KERNEL_TCGEN05, {}), id="tcgen05"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_FUSED_COMBINE": "1"}), id="tcgen05_fused"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_FUSED_COMBINE": "0"}), id="tcgen05_separate"),
           pytest.param((ops.KERNEL_TCGEN05, {"TT_TCGEN05_VARIANT": "3"}), id="tcgen05_2sm"),
           pytest.param((ops.KERNEL_MMA_SYNC, {}), id="mma_sync")]


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).cuda()


def host_cache(rng, B, Hkv, cap, D):
    """Random contents: codes without NaN, scales around 1 -> (k, ks, v, vs) uint8."""
    def one():
        c = rng.integers(0, 256, (B, Hkv, cap, D)).astype(np.uint8)
        c[(c & 127) == 127] = 0
        return c, rng.integers(118, 124, (B, Hkv, cap, D // 32)).astype(np.uint8)
    return (*one(), *one())


def device_cache(host):
    k, ks, v, vs = (u8(a) for a in host)
    return ops.MxCache(k, ks, v, vs)


def paged_cache(host, page_size, seed, lens, junk=255):
    """The same rows in shuffled pages; pages without a row below L_n are absent (-1), and every byte
    past L_n is junk (e4m3 NaN, scale 255)."""
    rng = np.random.default_rng(seed)
    B, Hkv, cap, _ = host[0].shape
    per = -(-cap // page_size)
    order = rng.permutation(B * per + 2)
    table = np.full((B, per), -1, dtype=np.int32)
    pools = [np.full((B * per + 2, Hkv, page_size, a.shape[3]), junk, dtype=np.uint8) for a in host]
    for n in range(B):
        for i in range(-(-int(lens[n]) // page_size)):
            table[n, i] = order[n * per + i]
            rows = min(page_size, int(lens[n]) - i * page_size)
            for pool, a in zip(pools, host):
                pool[table[n, i], :, :rows] = a[n, :, i * page_size:i * page_size + rows]
    k, ks, v, vs = (u8(p) for p in pools)
    return ops.MxCache(k, ks, v, vs, page_table=i32(table))


def tricky_rows(rng, B, T, Hkv, D):
    """bf16 rows over the format's corners: all magnitudes, zero blocks, ties, subnormals, infinities."""
    x = rng.standard_normal((B, T, Hkv, D)).astype(np.float32)
    x *= np.exp2(rng.integers(-140, 120, (B, T, Hkv, 1))).astype(np.float32)
    x[:, ::5] = np.exp2(rng.integers(-30, 30, x[:, ::5].shape)).astype(np.float32) * 1.0625
    x[:, 1::7, :, :32] = 0.0
    x[:, 2::7, :, 0] = np.inf
    x[:, 2::7, :, D - 1] = -np.inf
    return bf16_bits(x)


@pytest.mark.parametrize("advance", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,counts,lens", [
    (1, None, [0, 5, 39]), (16, [16, 0, 7], [0, 3, 33]), (40, [40, 1, 0], [0, 39, 40]), (5, [5, 5, 5], [35, 36, 0]),
    (3, [-1, 4, 2], [0, 0, -1]),
])
def test_append_bits(T, counts, lens, D, advance):
    rng = np.random.default_rng(T)
    B, Hkv, cap = 3, 2, 40
    host = host_cache(rng, B, Hkv, cap, D)
    cache = device_cache(host)
    new = [tricky_rows(rng, B, T, Hkv, D) for _ in range(2)]
    plan = ops.Plan(B, 2 * Hkv, Hkv, D, 4, ctx_capacity=cap)
    lens_d = i32(lens)
    for _ in range(2):   # twice: the write's block counter is back at zero
        lens_d.copy_(i32(lens))
        plan.kv_append_mx(dev(new[0]), dev(new[1]), cache, lens_d, i32(counts) if counts else None, advance=advance)
    want_counts = counts or [T] * B
    ref = [omx.kv_append_mx(f64(x), c, s, lens, want_counts, advance)
           for x, c, s in ((new[0], host[0], host[1]), (new[1], host[2], host[3]))]
    bad = ref[0][3]
    assert plan.check_status() == (ops.TT_ERR_DEVICE_ARG if bad.any() else ops.TT_OK)
    for got, want in ((cache.k, ref[0][0]), (cache.k_scale, ref[0][1]), (cache.v, ref[1][0]),
                      (cache.v_scale, ref[1][1]), (lens_d, ref[0][2])):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_append_nan_stays_in_its_element():
    x = np.ones((1, 1, 1, 64), dtype=np.float32)
    x[0, 0, 0, 3] = np.nan
    cache = ops.MxCache.empty(1, 1, 8, 64)
    plan = ops.Plan(1, 1, 1, 64, 1, ctx_capacity=8)
    lens = i32([2])
    plan.kv_append_mx(dev(bf16_bits(x)), dev(bf16_bits(x)), cache, lens)
    out = [torch.full((1, 1, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plan.kv_read_mx(cache, lens, i32([2]), *out)
    plan.check()
    for o in out:
        o = o.float().cpu().numpy()[0, 0, 0]
        assert np.isnan(o[3]) and (np.delete(o, 3) == 1.0).all()


@pytest.mark.parametrize("page_size", [0, 16, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_read_back_exactly(D, page_size):
    rng = np.random.default_rng(7)
    B, Hkv, cap, T = 4, 3, 50, 20
    lens, starts = [50, 0, 17, 31], [30, 0, 5, 40]
    host = host_cache(rng, B, Hkv, cap, D)
    for s in host[1::2]:
        s[:] = rng.integers(0, 247, s.shape)      # every scale below overflow, down to bf16's subnormals
    cache = paged_cache(host, page_size, 8, lens) if page_size else device_cache(host)
    plan = ops.Plan(B, Hkv, Hkv, D, 1, ctx_capacity=cap)
    out = [torch.full((B, Hkv, T, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plan.kv_read_mx(cache, i32(lens), i32(starts), *out)
    plan.check()
    for o, c, s in ((out[0], host[0], host[1]), (out[1], host[2], host[3])):
        ref = omx.kv_read_mx(c, s, lens, starts, np.full((B, Hkv, T, D), 3.0))
        want = torch.from_numpy(ref).to(torch.bfloat16)     # rounds the values below bf16's subnormals
        assert torch.equal(o.cpu(), want)


def test_read_back_flags_what_it_cannot_read():
    cache = ops.MxCache.empty(2, 1, 8, 64)
    plan = ops.Plan(2, 1, 1, 64, 1, ctx_capacity=8)
    out = [torch.full((2, 1, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plan.kv_read_mx(cache, i32([8, 8]), i32([-1, 6]), *out)
    assert plan.check_status() == ops.TT_ERR_DEVICE_ARG
    for o in out:
        assert (o[0] == 3).all() and not o[1, :, :2].any() and (o[1, :, 2:] == 3).all()
    plan.kv_read_mx(cache, i32([9, -2]), i32([0, 0]), *out)
    assert plan.check_status() == ops.TT_ERR_DEVICE_ARG


@pytest.mark.parametrize("page_size", [16, 32])
def test_append_into_pages(page_size):
    rng = np.random.default_rng(9)
    B, Hkv, D, cap, T = 3, 2, 64, 96, 30
    lens, counts = [10, 50, 0], [30, 17, 29]
    ends = [a + b for a, b in zip(lens, counts)]
    host = host_cache(rng, B, Hkv, cap, D)
    cache = paged_cache(host, page_size, 10, ends)
    new = [tricky_rows(rng, B, T, Hkv, D) for _ in range(2)]
    plan = ops.Plan(B, Hkv, Hkv, D, 1)
    lens_d = i32(lens)
    plan.kv_append_mx(dev(new[0]), dev(new[1]), cache, lens_d, i32(counts))
    plan.check()
    assert lens_d.tolist() == ends
    table = cache.page_table.cpu().numpy()
    for got, gots, x, c, s in ((cache.k, cache.k_scale, new[0], host[0], host[1]),
                               (cache.v, cache.v_scale, new[1], host[2], host[3])):
        rc, rs, _, _ = omx.kv_append_mx(f64(x), c, s, lens, counts)
        got, gots = got.cpu().numpy(), gots.cpu().numpy()
        for n in range(B):
            for pos in range(ends[n]):
                pg = table[n, pos // page_size]
                np.testing.assert_array_equal(got[pg, :, pos % page_size], rc[n, :, pos])
                np.testing.assert_array_equal(gots[pg, :, pos % page_size], rs[n, :, pos])
    cache.page_table[0, 1] = 10 ** 6
    lens_d.copy_(i32(lens))
    plan.kv_append_mx(dev(new[0]), dev(new[1]), cache, lens_d, i32(counts))
    assert plan.check_status() == ops.TT_ERR_DEVICE_ARG


def check_attention(inp, host, out, lse, window=0, sinks=0, parents=None, what=""):
    kc, vc = omx.values(host[0], host[1]), omx.values(host[2], host[3])
    ro, rl = vis.block_attn_visible(f64(inp.q), kc, vc, f64(inp.k_blk), f64(inp.v_blk), inp.ctx_lens, window, sinks,
                                    parents)
    gone = np.isinf(rl)
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), gone), what
    assert_parity(out, ro, f"{what} out")
    assert_parity(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse), np.where(gone, 0.0, rl), f"{what} lse")


def attention_case(shape, seed):
    B, S, Hq, Hkv, D, Lcap, lens = SHAPES[shape]
    inp = make_decode(B, S, Hq, Hkv, D, Lcap, seed=seed, ctx_lens=lens)
    rng = np.random.default_rng(seed)
    q = [omx.quantise(f64(x)) for x in (inp.k_ctx, inp.v_ctx)]
    host = (*q[0], *q[1])
    junk = tuple(a.copy() for a in host)
    for n, L in enumerate(lens):
        for a in junk:
            a[n, :, L:] = 255
    return (B, S, Hq, Hkv, D, Lcap, lens), inp, host, junk, rng


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (130, 70), (1, 0)])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_attention(shape, window, sinks, tree, kernel):
    (B, S, Hq, Hkv, D, Lcap, lens), inp, host, junk, rng = attention_case(shape, 80)
    par = tree_cases(B, S, rng) if tree else None
    q, kb, vb = poison_absent(inp, par) if tree else (inp.q, inp.k_blk, inp.v_blk)
    plan = make_plan(kernel, B, Hq, Hkv, D, S, ctx_capacity=Lcap, window=window, sinks=sinks)
    out, lse = plan.block_attn_mx(dev(q), device_cache(junk), dev(kb), dev(vb), i32(lens),
                                  parents=i32(par) if tree else None, want_lse=True)
    plan.check()
    check_attention(inp, host, out, lse, window, sinks, par, f"{shape} W={window}")


@pytest.mark.parametrize("kernel", [KERNELS[0], KERNELS[1], KERNELS[4]])
@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks,tree", [(0, 0, False), (0, 0, True), (100, 4, False), (130, 70, True)])
@pytest.mark.parametrize("shape", ["S16-g16", "S1-g16", "S5-g3-d64", "S64-g4"])
def test_attention_paged(shape, window, sinks, tree, page_size, kernel):
    (B, S, Hq, Hkv, D, Lcap, lens), inp, host, _, rng = attention_case(shape, 81)
    par = tree_cases(B, S, rng) if tree else None
    q, kb, vb = poison_absent(inp, par) if tree else (inp.q, inp.k_blk, inp.v_blk)
    plan = make_plan(kernel, B, Hq, Hkv, D, S, window=window, sinks=sinks)
    out, lse = plan.block_attn_mx(dev(q), paged_cache(host, page_size, 82, lens), dev(kb), dev(vb), i32(lens),
                                  parents=i32(par) if tree else None, want_lse=True)
    plan.check()
    check_attention(inp, host, out, lse, window, sinks, par, f"{shape} P={page_size}")


@pytest.mark.parametrize("num_ctas", [1, 3, 37, 148, 300])
def test_attention_split_invariance(num_ctas):
    (B, S, Hq, Hkv, D, Lcap, lens), inp, host, junk, _ = attention_case("S16-g16", 83)
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap, num_ctas=num_ctas)
    out, lse = plan.block_attn_mx(dev(inp.q), device_cache(junk), dev(inp.k_blk), dev(inp.v_blk), i32(lens),
                                  want_lse=True)
    plan.check()
    check_attention(inp, host, out, lse, what=f"C={num_ctas}")


@pytest.mark.parametrize("big", [2.0 ** 20, 2.0 ** -60])
def test_attention_with_far_scales(big):
    """Values far from 1 (scale bytes whose power of two, times the format's offset, leaves bf16): the
    queries carry the inverse factor, so the scores are ordinary; V's factor divides out of the check."""
    (B, S, Hq, Hkv, D, Lcap, lens), inp, host, _, _ = attention_case("S5-g3-d64", 84)
    shift = int(np.log2(big))
    far = (host[0], (host[1].astype(int) + shift).astype(np.uint8), host[2], (host[3].astype(int) + shift).astype(np.uint8))
    q = bf16_bits((f64(inp.q) / big).astype(np.float32))
    inp.q = q
    inp.k_blk = bf16_bits((f64(inp.k_blk) * big).astype(np.float32))
    inp.v_blk = bf16_bits((f64(inp.v_blk) * big).astype(np.float32))
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap)
    out, lse = plan.block_attn_mx(dev(q), device_cache(far), dev(inp.k_blk), dev(inp.v_blk), i32(lens), want_lse=True)
    plan.check()
    kc, vc = omx.values(far[0], far[1]), omx.values(far[2], far[3])
    ro, rl = vis.block_attn_visible(f64(q), kc, vc, f64(inp.k_blk), f64(inp.v_blk), lens)
    assert_parity(out.double() / big, ro / big, "out")
    assert_parity(lse, rl, "lse")


def test_serving_run_write_attend_commit_read():
    """The operators together, as a serving loop uses them: a prompt is written, a drafted tree is verified
    over the cache, its accepted rows are committed (ragged counts), the next block attends, and the
    cache is read back into the bf16 slab that the plain attention gives the same answer over."""
    rng = np.random.default_rng(90)
    B, S, Hq, Hkv, D, cap = 4, 8, 8, 2, 128, 300
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=cap)
    cache = ops.MxCache.empty(B, Hkv, cap, D)
    lens_d = i32([0] * B)
    lens = np.zeros(B, dtype=np.int64)
    host = [np.zeros((B, Hkv, cap, D), np.uint8), np.zeros((B, Hkv, cap, D // 32), np.uint8)] * 2

    def rows(T, heads=Hkv):
        return bf16_bits(rng.standard_normal((B, T, heads, D)).astype(np.float32))

    def append(T, counts):
        nonlocal lens, host
        k, v = rows(T), rows(T)
        plan.kv_append_mx(dev(k), dev(v), cache, lens_d, i32(counts))
        kc, ks, new, _ = omx.kv_append_mx(f64(k), host[0], host[1], lens, counts)
        vc, vs, new, _ = omx.kv_append_mx(f64(v), host[2], host[3], lens, counts)
        host, lens = [kc, ks, vc, vs], new

    append(200, [200, 1, 0, 77])
    for step in range(3):
        inp = make_decode(B, S, Hq, Hkv, D, cap, seed=91 + step, ctx_lens=list(lens))
        par = tree_cases(B, S, rng)
        q, kb, vb = poison_absent(inp, par)
        out, lse = plan.block_attn_mx(dev(q), cache, dev(kb), dev(vb), lens_d, parents=i32(par), want_lse=True)
        check_attention(inp, host, out, lse, parents=par, what=f"step {step}")
        append(S, [8, 3, 0, 5])
    assert lens_d.tolist() == list(lens)
    inp = make_decode(B, S, Hq, Hkv, D, cap, seed=99, ctx_lens=list(lens))
    x = dev(inp.q), dev(inp.k_blk), dev(inp.v_blk)
    out = plan.block_attn_mx(x[0], cache, x[1], x[2], lens_d)
    kc, vc = (torch.zeros((B, Hkv, cap, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    plan.kv_read_mx(cache, lens_d, None, kc, vc)
    plain = plan.block_attn(x[0], kc, vc, x[1], x[2], lens_d)
    plan.check()
    # the same bf16 operands in both calls; weights may round differently where the exp2 differs
    assert float((out - plain).abs().max()) <= 2.0 ** -8 * 4


def test_in_a_graph_on_another_stream():
    """append, attention and read-back captured once and replayed: lengths advance on the device."""
    (B, S, Hq, Hkv, D, Lcap, _), inp, host, _, rng = attention_case("S5-g3-d64", 95)
    lens = [100, 40, 0]
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=Lcap)
    cache = device_cache(host)
    lens_d, lens0 = i32(lens), i32(lens)
    new = [dev(bf16_bits(rng.standard_normal((B, S, Hkv, D)).astype(np.float32))) for _ in range(2)]
    x = [dev(t) for t in (inp.q, inp.k_blk, inp.v_blk)]
    out = torch.empty((B, S, Hq, D), device="cuda")
    back = [torch.zeros((B, Hkv, Lcap, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def calls():
        plan.kv_append_mx(new[0], new[1], cache, lens_d)
        plan.block_attn_mx(x[0], cache, x[1], x[2], lens_d, out=out)
        plan.kv_read_mx(cache, lens_d, None, *back)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            calls()
        lens_d.copy_(lens0)
        for _ in range(3):
            g.replay()
        side.synchronize()
        assert lens_d.tolist() == [a + 3 * S for a in lens]
        want = plan.block_attn(x[0], back[0], back[1], x[1], x[2], lens_d)
        side.synchronize()
        assert float((out - want).abs().max()) <= 2.0 ** -8 * 4
    plan.check()
