"""CPU pins of the oracles for windows, sinks, drafted trees and the microscaled cache."""
import numpy as np
import pytest
import torch

from oracle import block_attn, block_causal, block_causal_backward
from oracle import mx as omx
from oracle import visibility as vis


def rand(rng, *shape):
    return rng.standard_normal(shape)


def test_window_by_an_explicit_predicate():
    for L in (0, 1, 5, 9, 30):
        for w, s in ((1, 0), (4, 2), (9, 3), (30, 1), (7, 40)):
            want = [c for c in range(L) if c < s or L - c <= w]
            assert list(np.flatnonzero(vis.visible_context(L, w, s))) == want


def test_no_window_and_no_tree_is_the_plain_oracle():
    rng = np.random.default_rng(0)
    q, kb, vb = rand(rng, 2, 4, 4, 8), rand(rng, 2, 4, 2, 8), rand(rng, 2, 4, 2, 8)
    kc, vc = rand(rng, 2, 2, 9, 8), rand(rng, 2, 2, 9, 8)
    o, l = vis.block_attn_visible(q, kc, vc, kb, vb, [9, 3])
    ro, rl = block_attn(q, kc, vc, kb, vb, [9, 3])
    np.testing.assert_allclose(o, ro, atol=1e-13)
    np.testing.assert_allclose(l, rl, atol=1e-13)


def test_tree_against_torch_sdpa_with_the_mask():
    """A tree's rows against torch's float64 attention with an explicitly built ancestor mask."""
    rng = np.random.default_rng(1)
    S, L, D = 7, 5, 8
    par = [-1, 0, 0, 2, -1, 4, 2]
    paths = {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 2, 3], 4: [4], 5: [4, 5], 6: [0, 2, 6]}
    q, kb, vb = rand(rng, 1, S, 2, D), rand(rng, 1, S, 1, D), rand(rng, 1, S, 1, D)
    kc, vc = rand(rng, 1, 1, L, D), rand(rng, 1, 1, L, D)
    mask = torch.zeros(S, L + S, dtype=torch.bool)
    mask[:, :L] = True
    for t, p in paths.items():
        mask[t, [L + u for u in p]] = True
    k = torch.from_numpy(np.concatenate([kc[0, 0], kb[0, :, 0]]))
    v = torch.from_numpy(np.concatenate([vc[0, 0], vb[0, :, 0]]))
    o, _ = vis.block_attn_visible(q, kc, vc, kb, vb, [L], parents=[par])
    for j in range(2):
        ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[0, :, j])[None], k[None], v[None],
                                                               attn_mask=mask)[0]
        np.testing.assert_allclose(o[0, :, j], ref.numpy(), atol=1e-13)


def test_absent_rows_and_their_descendants_see_nothing():
    sees, there = vis.tree_visibility([-1, -2, 1, 0, 2])
    assert list(there) == [True, False, False, True, False]
    assert not sees[[1, 2, 4]].any() and list(np.flatnonzero(sees[3])) == [0, 3]
    rng = np.random.default_rng(2)
    q, kb, vb = rand(rng, 1, 2, 1, 8), rand(rng, 1, 2, 1, 8), rand(rng, 1, 2, 1, 8)
    kc = rand(rng, 1, 1, 3, 8)
    o, l = vis.block_attn_visible(q, kc, kc, kb, vb, [3], parents=[[-2, -1]])
    assert not o[0, 0].any() and l[0, 0, 0] == -np.inf and np.isfinite(l[0, 0, 1])


def test_causal_window_wide_enough_is_block_causal_with_its_backward():
    rng = np.random.default_rng(3)
    B, N, S, Hq, Hkv, D = 1, 12, 3, 4, 2, 8
    q, do = rand(rng, B, N, Hq, D), rand(rng, B, N, Hq, D)
    kc, vc = rand(rng, B, Hkv, N, D), rand(rng, B, Hkv, N, D)
    kb, vb = rand(rng, B, N, Hkv, D), rand(rng, B, N, Hkv, D)
    o, l = vis.block_causal_window(q, kc, vc, kb, vb, S, N, 0)
    ro, rl = block_causal(q, kc, vc, kb, vb, S)
    np.testing.assert_allclose(o, ro, atol=1e-13)
    np.testing.assert_allclose(l, rl, atol=1e-13)
    for a, b in zip(vis.block_causal_window_backward(q, kc, vc, kb, vb, do, S, N, 0),
                    block_causal_backward(q, kc, vc, kb, vb, do, S)):
        np.testing.assert_allclose(a, b, atol=1e-12)


def test_window_backward_by_differences():
    """Central differences: error ~ h^2 |f'''| + eps |f| / h ~ 1e-10 + 1e-10 at h = 1e-5; bar 1e-7."""
    rng = np.random.default_rng(4)
    B, N, S, Hq, Hkv, D = 1, 8, 2, 2, 1, 4
    w, sinks, h = 3, 1, 1e-5
    x = dict(q=rand(rng, B, N, Hq, D), k_ctx=rand(rng, B, Hkv, N, D), v_ctx=rand(rng, B, Hkv, N, D),
             k_blk=rand(rng, B, N, Hkv, D), v_blk=rand(rng, B, N, Hkv, D))
    do = rand(rng, B, N, Hq, D)

    def f(**kw):
        return (do * vis.block_causal_window(**{**x, **kw}, block_size=S, window=w, sinks=sinks)[0]).sum()

    grads = vis.block_causal_window_backward(**x, dout=do, block_size=S, window=w, sinks=sinks)
    for name, gr in zip(("q", "k_blk", "v_blk"), grads):
        for i in range(0, x[name].size, 5):
            d = np.zeros(x[name].size)
            d[i] = h
            d = d.reshape(x[name].shape)
            num = (f(**{name: x[name] + d}) - f(**{name: x[name] - d})) / (2 * h)
            assert abs(num - gr.ravel()[i]) < 1e-7


def test_mx_codes_against_torch_e4m3():
    """Every e4m3 code and the halfway points between neighbours, against torch's own conversion."""
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(np.isnan(ref), np.isnan(omx.E4M3))
    np.testing.assert_array_equal(ref[~np.isnan(ref)], omx.E4M3[~np.isnan(ref)])
    pos = omx.E4M3[:127]
    y = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, -(pos[1:] + pos[:-1]) / 2])
    y = np.concatenate([y, np.zeros(-len(y) % 31)]).reshape(-1, 31)
    y = np.concatenate([y, np.full((len(y), 1), 448.0)], axis=1)      # fixes the scale at 1
    c, s = omx.quantise(y)
    assert (s == 127).all()
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(c, want)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.5, 1), (449.0, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7),
                                    (2.0 ** -133, -127), (0.0, -127), (3.38e38, 120)])
def test_mx_scale_is_the_least_that_holds_amax(amax, e):
    x = np.zeros(32)
    x[7] = -amax
    c, s = omx.quantise(x)
    assert int(s[0]) - 127 == e
    v = omx.values(c, s)
    assert v[7] <= 0 and abs(v[7] + amax) <= max(abs(amax) * 2.0 ** -4, 2.0 ** -137)


def test_mx_nonfinite_and_roundtrip():
    x = np.zeros(64)
    x[:4] = [np.inf, -np.inf, np.nan, 3.0]
    c, s = omx.quantise(x)
    v = omx.values(c, s)
    top = 448.0 * 2.0 ** (int(s[0]) - 127)
    assert v[0] == top and v[1] == -top and np.isnan(v[2]) and v[3] == 3.0 and not v[32:].any()
    rng = np.random.default_rng(5)
    c = rng.integers(0, 127, (9, 64)).astype(np.uint8)
    c[:, ::32] = 126                                             # every block reaches 448
    s = rng.integers(0, 240, (9, 2)).astype(np.uint8)
    c2, s2 = omx.quantise(omx.values(c, s))
    np.testing.assert_array_equal(c, c2)
    np.testing.assert_array_equal(s, s2)
