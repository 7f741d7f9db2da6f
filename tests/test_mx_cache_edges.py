"""The quantised cache at its edges: the alignment of its scale copies, and pages outside the pool."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from oracle import visibility as vis
from two_tower_block_b200 import ops


def _scale_word_cases(rng):
    for D in (64, 128):
        for page in (0, 16, 32, 64, 128, 65536):
            for count in (1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64):
                for _ in range(6):
                    if page == 0:
                        yield D, page, [int(rng.integers(0, 1 << 30))], count
                    else:
                        sub = min(page, 64)
                        n = 64 // sub
                        rows = [int(rng.integers(0, (1 << 30) // sub)) * sub for _ in range(n)]
                        yield D, page, [r if rng.random() < 0.6 else -1 for r in rows], count
    for page in (16, 32):   # a page outside the pool in front of pages inside it
        yield 64, page, [-1] + [page * (7 + i) for i in range(64 // page - 1)], 64


def test_scale_copies_are_aligned_and_bring_every_row():
    """Each copy is of at most four bytes from a multiple of four, as the asynchronous copy demands; every
    row inside the pool finds all of its scale bytes where the converters read them; no byte outside the
    tile's rows is copied but those of the row in front of an odd one."""
    rng = np.random.default_rng(3)
    for D, page, rows, count in _scale_word_cases(rng):
        per = D // 32
        sub = 64 if page == 0 else min(page, 64)
        words, first = ops.mx_scale_words(D, page, rows, count)
        got = {}
        for to, at, num in words:
            assert at >= 0 and at % 4 == 0 and to % 4 == 0 and 0 < num <= 4, (D, page, rows, count)
            got.update({to + i: at + i for i in range(num)})
        want = {}
        for r in range(count):
            base = rows[r // sub]
            if base >= 0:
                for i in range(per):
                    want[first + r * per + i] = (base + r % sub) * per + i
        assert {k: got.get(k) for k in want} == want, (D, page, rows, count)
        extra = set(got) - set(want)
        assert extra <= set(range(first)), (D, page, rows, count)


def test_scale_copies_refuse_bad_arguments():
    for args in ((96, 0, [0], 1), (64, 24, [0], 1), (64, 0, [0], 0), (64, 0, [0], 65)):
        with pytest.raises(ops.TTError) as e:
            ops.mx_scale_words(*args)
        assert e.value.status == ops.TT_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [ops.KERNEL_TCGEN05, ops.KERNEL_MMA_SYNC])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 20)])
@pytest.mark.parametrize("page_size", [16, 32, 64])
@pytest.mark.parametrize("S,g,D", [(5, 3, 64), (16, 16, 64), (16, 16, 128), (1, 16, 128)])
def test_pages_outside_the_pool_read_as_zeros(S, g, D, page_size, window, sinks, kernel):
    from tests.gpu_util import assert_parity, dev, f64
    from tests.test_parity_mx import i32, paged_cache
    from two_tower_block_b200.workloads import make_decode
    B, Hkv, cap, lens = 3, 2, 192, [192, 75, 129]
    inp = make_decode(B, S, g * Hkv, Hkv, D, cap, seed=41, ctx_lens=lens)
    q = [omx.quantise(f64(x)) for x in (inp.k_ctx, inp.v_ctx)]
    host = [a.copy() for a in (*q[0], *q[1])]
    cache = paged_cache(host, page_size, 42, lens)
    bad = [(0, 0, -1), (0, 64 // page_size, 10 ** 6), (0, 128 // page_size, -7), (1, 0, cache.shape[0]), (2, 1, -1)]
    for n, i, page in bad:
        cache.page_table[n, i] = page
        for a in host:
            a[n, :, i * page_size:(i + 1) * page_size] = 0     # what such a page reads as: values 0 * 2^-127
    plan = ops.Plan(B, g * Hkv, Hkv, D, S, window=window, sinks=sinks, kernel=kernel)
    out, lse = plan.block_attn_mx(dev(inp.q), cache, dev(inp.k_blk), dev(inp.v_blk), i32(lens), want_lse=True)
    assert plan.check_status() == ops.TT_ERR_DEVICE_ARG
    ro, rl = vis.block_attn_visible(f64(inp.q), omx.values(host[0], host[1]), omx.values(host[2], host[3]),
                                    f64(inp.k_blk), f64(inp.v_blk), lens, window, sinks)
    assert_parity(out, ro, "out")
    assert_parity(lse, rl, "lse")


@pytest.mark.parametrize("shape", [(2, 0), (0, 0)])
def test_a_table_without_entries_is_no_slab(shape):
    """Pages without a single table entry hold no position; without an address for the table the library would
    take the pools for slabs of the plan's capacity."""
    values, scales = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 16, 2, dtype=torch.uint8)
    table = torch.zeros(shape, dtype=torch.int32)
    cache = ops.MxCache(values, scales, values.clone(), scales.clone(), page_table=table)
    assert cache._d.page_table and cache._d.page_table % 4 == 0
    assert (cache._d.num_pages, cache._d.page_size, cache._d.pages_per_seq) == (3, 16, 0)
    assert ops.MxCache(values, scales, values.clone(), scales.clone())._d.page_table is None


@pytest.mark.parametrize("name", ["k", "k_scale", "v", "v_scale", "page_table"])
def test_a_cache_keeps_its_tensors(name):
    """The calls use the addresses taken when the cache was made: another tensor put in its place would be
    ignored, and the old one's memory could go to someone else."""
    values, scales = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 16, 2, dtype=torch.uint8)
    cache = ops.MxCache(values, scales, values.clone(), scales.clone(), page_table=torch.zeros(2, 4, dtype=torch.int32))
    old = getattr(cache, name)
    with pytest.raises(AttributeError):
        setattr(cache, name, old.clone())
    assert getattr(cache, name) is old


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [ops.KERNEL_TCGEN05, ops.KERNEL_MMA_SYNC])
def test_a_cache_without_positions(kernel):
    from tests.gpu_util import assert_parity, dev, f64
    from tests.test_parity_mx import i32
    from two_tower_block_b200.workloads import make_decode
    B, S, Hq, Hkv, D = 2, 5, 6, 2, 64
    inp = make_decode(B, S, Hq, Hkv, D, 40, seed=43, ctx_lens=[0, 0])
    table = torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    cache = ops.MxCache.empty(1, Hkv, 16, D, page_table=table)
    plan = ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=4096, kernel=kernel)   # a capacity that the pool does not hold
    x = dev(inp.q), dev(inp.k_blk), dev(inp.v_blk)
    ro, rl = vis.block_attn_visible(f64(inp.q), f64(inp.k_ctx), f64(inp.v_ctx), f64(inp.k_blk), f64(inp.v_blk), [0, 0])
    for lens, status in (([0, 0], ops.TT_OK), ([0, 30], ops.TT_ERR_DEVICE_ARG)):   # 30: clamped to 0
        out, lse = plan.block_attn_mx(x[0], cache, x[1], x[2], i32(lens), want_lse=True)
        assert plan.check_status() == status
        assert_parity(out, ro, "out")
        assert_parity(lse, rl, "lse")
    lens = i32([0, 0])
    plan.kv_append_mx(x[1], x[2], cache, lens)
    assert plan.check_status() == ops.TT_ERR_DEVICE_ARG and lens.tolist() == [0, 0]
    assert not cache.k.view(torch.uint8).any() and not cache.k_scale.any()
    back = [torch.full((B, Hkv, 3, D), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plan.kv_read_mx(cache, lens, None, *back)
    plan.check()
    assert all((b == 2).all() for b in back)
