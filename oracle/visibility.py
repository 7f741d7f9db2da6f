"""Float64 CPU oracle of block attention with a sliding window, first tokens that stay visible
(sinks), and drafted trees.

TEST INFRASTRUCTURE ONLY (same rule as ``oracle.oracle``).

What it computes: the attention of ``oracle.oracle`` with the key set written as a boolean matrix.
Of the L committed positions in front of a block, position c is visible when c < sinks or
c >= L - window (window 0: all of them).  In a tree, block row t sees block row u when u is t or an
ancestor of t; a row that is absent (-2), or has an absent ancestor, sees nothing, context included:
its output is 0 and its lse -inf.
"""
from __future__ import annotations

import numpy as np

__all__ = ["visible_context", "tree_visibility", "block_attn_visible", "block_causal_window",
           "block_causal_window_backward"]


def visible_context(L, window, sinks):
    """Boolean [L]: which committed positions a block at L sees."""
    c = np.arange(L)
    return np.ones(L, dtype=bool) if window == 0 else (c < sinks) | (c >= L - window)


def tree_visibility(parents):
    """Boolean [S, S] and [S]: what each row of one tree sees of the block, and which rows are there."""
    S = len(parents)
    sees = np.zeros((S, S), dtype=bool)
    there = np.zeros(S, dtype=bool)
    for t in range(S):
        p = int(parents[t])
        if p == -1:
            there[t] = True
        elif 0 <= p < t:
            there[t] = there[p]
            sees[t] = sees[p]
        if there[t]:
            sees[t, t] = True
        else:
            sees[t] = False
    return sees, there


def _attend(q, keys, vals, sees, scale):
    """Rows q [R, D] over the keys that sees [R, K] allows: (out, lse, weights)."""
    out = np.zeros((q.shape[0], vals.shape[1]))
    lse = np.full(q.shape[0], -np.inf)
    w = np.zeros(sees.shape)
    for r in range(q.shape[0]):
        k = np.flatnonzero(sees[r])
        if k.size == 0:
            continue
        s = scale * (keys[k] @ q[r])
        m = s.max()
        e = np.exp(s - m)
        w[r, k] = e / e.sum()
        out[r] = w[r, k] @ vals[k]
        lse[r] = m + np.log(e.sum())
    return out, lse, w


def block_attn_visible(q, k_ctx, v_ctx, k_blk, v_blk, ctx_lens, window=0, sinks=0, parents=None, scale=None):
    """Decode (shapes of oracle.block_attn, float64) with a window and/or a tree [B, S]."""
    B, S, Hq, D = q.shape
    Hkv = k_blk.shape[2]
    g = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out = np.zeros((B, S, Hq, D))
    lse = np.full((B, Hq, S), -np.inf)
    for n in range(B):
        L = int(ctx_lens[n])
        c = np.flatnonzero(visible_context(L, window, sinks))
        sees, there = (np.ones((S, S), dtype=bool), np.ones(S, dtype=bool)) if parents is None \
            else tree_visibility(parents[n])
        rows = np.flatnonzero(there)
        if rows.size == 0:
            continue
        vis = np.concatenate([np.ones((rows.size, c.size), dtype=bool), sees[np.ix_(rows, rows)]], axis=1)
        for h in range(Hkv):
            keys = np.concatenate([k_ctx[n, h][c], k_blk[n, rows, h]])
            vals = np.concatenate([v_ctx[n, h][c], v_blk[n, rows, h]])
            for j in range(h * g, (h + 1) * g):
                o, l, _ = _attend(q[n, rows, j], keys, vals, vis, scale)
                out[n, rows, j] = o
                lse[n, j, rows] = l
    return out, lse


def _block(q, k_ctx, v_ctx, k_blk, v_blk, n, h, b, S, window, sinks):
    lo = S * b
    c = np.flatnonzero(visible_context(lo, window, sinks))
    keys = np.concatenate([k_ctx[n, h][c], k_blk[n, lo:lo + S, h]])
    vals = np.concatenate([v_ctx[n, h][c], v_blk[n, lo:lo + S, h]])
    return lo, keys, vals


def block_causal_window(q, k_ctx, v_ctx, k_blk, v_blk, block_size, window, sinks, scale=None):
    """Whole sequences (shapes of oracle.block_causal): block b is the decode with L = S*b."""
    B, N, Hq, D = q.shape
    S = block_size
    out = np.zeros((B, N, Hq, D))
    lse = np.zeros((B, Hq, N))
    for b in range(N // S):
        sl = slice(S * b, S * b + S)
        out[:, sl], lse[:, :, sl] = block_attn_visible(q[:, sl], k_ctx, v_ctx, k_blk[:, sl], v_blk[:, sl],
                                                       [S * b] * B, window, sinks, scale=scale)
    return out, lse


def block_causal_window_backward(q, k_ctx, v_ctx, k_blk, v_blk, dout, block_size, window, sinks, scale=None):
    """Gradients (dq, dk_blk, dv_blk) of sum(dout * out) of block_causal_window."""
    B, N, Hq, D = q.shape
    Hkv = k_blk.shape[2]
    g, S = Hq // Hkv, block_size
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    dq = np.zeros(q.shape)
    dk, dv = np.zeros(k_blk.shape), np.zeros(v_blk.shape)
    for n in range(B):
        for h in range(Hkv):
            for b in range(N // S):
                lo, keys, vals = _block(q, k_ctx, v_ctx, k_blk, v_blk, n, h, b, S, window, sinks)
                for j in range(h * g, (h + 1) * g):
                    qr, do = q[n, lo:lo + S, j], dout[n, lo:lo + S, j]
                    o, _, p = _attend(qr, keys, vals, np.ones((S, len(keys)), dtype=bool), scale)
                    ds = p * (do @ vals.T - (do * o).sum(axis=1, keepdims=True))
                    dq[n, lo:lo + S, j] = scale * ds @ keys
                    dk[n, lo:lo + S, h] += scale * ds[:, -S:].T @ qr
                    dv[n, lo:lo + S, h] += p[:, -S:].T @ do
    return dq, dk, dv
