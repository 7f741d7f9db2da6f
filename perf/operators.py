"""The serving and training operators around the block attention, as one measured set.

Four operators, each in its plain form (elementary torch operations in 32 bits, rounded once) and
through this repository's public calls:

* ``window``  block attention whose context is a sliding window and a few first tokens (sinks):
  decode over a contiguous or a paged cache;
* ``train``   the same visibility over whole sequences, forward and backward;
* ``tree``    block attention whose block is a tree of drafted tokens (a node sees the whole
  context, its ancestors and itself), over a contiguous or a paged cache;
* ``cache``   a context cache in microscaled e4m3 (one power-of-two scale per 32 elements): the new
  rows are quantised as they are written, and rows are read back;
* ``mx``      block attention over that cache, for a denoiser's block, a tree or a single token.
"""
import functools
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one token per sequence on a windowed layer: the smallest call of a decode loop
        dict(name="window_token", op="window", B=8, S=1, Hq=32, Hkv=2, D=128, cap=4096, ragged=False, page=0,
             window=1024, sinks=4),
        # a serving batch of 16-token blocks with widely different contexts, from 64-row pages
        dict(name="window_ragged_paged", op="window", B=64, S=16, Hq=32, Hkv=2, D=128, cap=16384, ragged=True,
             page=64, window=2000, sinks=16),
        # a small training step of a windowed layer with an odd window
        dict(name="train_small", op="train", B=2, N=1000, S=8, Hq=8, Hkv=2, D=64, window=250, sinks=3),
        # the training workload's shape at half its batch: forward and backward of a windowed layer
        dict(name="train_8192", op="train", B=4, N=8192, S=16, Hq=32, Hkv=2, D=128, window=1024, sinks=16),
        # one sequence, few drafted tokens, a short context
        dict(name="tree_small", op="tree", B=1, S=8, Hq=4, Hkv=1, D=64, cap=256, ragged=False, page=0),
        # a batch that verifies 16 drafted tokens per sequence
        dict(name="tree_16", op="tree", B=8, S=16, Hq=32, Hkv=2, D=128, cap=4096, ragged=False, page=0),
        # wide trees (64 nodes) over ragged contexts in pages
        dict(name="tree_64_paged", op="tree", B=16, S=64, Hq=8, Hkv=2, D=128, cap=8192, ragged=True, page=32),
        # a committed 16-token block: write it, read the cache's tail back
        dict(name="cache_block", op="cache", B=8, T=16, Hkv=2, D=128, cap=4096, held=4000, rows=256),
        # whole prompts written into an empty cache and read back
        dict(name="cache_prompt", op="cache", B=4, T=131000, Hkv=2, D=128, cap=131072, held=0, rows=131072),
        # one token per sequence over a quantised cache
        dict(name="mx_token", op="mx", B=8, S=1, Hq=32, Hkv=2, D=128, cap=4096, ragged=False, page=0, tree=False),
        # the ragged serving batch over a quantised paged cache, with drafted trees
        dict(name="mx_ragged_paged", op="mx", B=64, S=16, Hq=32, Hkv=2, D=128, cap=16384, ragged=True, page=64,
             tree=True),
        # the longest contexts: 16-token blocks over 131072 committed tokens
        dict(name="mx_long", op="mx", B=4, S=16, Hq=32, Hkv=2, D=128, cap=131072, ragged=False, page=0, tree=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: the same operators over batch 1 to 64, 1 to 64 block tokens, one to 16 query
    heads per KV head, both head sizes, contexts of one to 131072 tokens."""
    op = rng.choice(["window", "train", "tree", "cache", "mx"])
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    g = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "cache":
        cap = _log_int(rng, 16, 131072)
        B = max(1, min(_log_int(rng, 1, 64), (1 << 27) // (cap * Hkv * D)))
        T = _log_int(rng, 1, cap)
        return dict(op=op, B=B, T=T, Hkv=Hkv, D=D, cap=cap, held=rng.randint(0, cap - T), rows=_log_int(rng, 1, cap))
    if op == "train":
        S = rng.choice([1, 4, 5, 8, 16, 32])
        S = max(1, min(S, 256 // g))
        N = S * _log_int(rng, 4, max(5, 8192 // S))
        window = _log_int(rng, 8, 1024)
        B = max(1, min(_log_int(rng, 1, 8), (4 * 8192 * 32 * 1024) // (N * g * Hkv * (window + 64))))
        while B * N * g * Hkv > 4 * 8192 * 32 or B * N * g * Hkv * (window + 32 + S) > 4 * 8192 * 32 * 1056 or \
                B * (N // S) * Hkv * (window + 32 + S) > 4 * 512 * 2 * 8 * 1056:
            N = S * max(2, N // S // 2)
            if N == 2 * S:
                B = max(1, B // 2)
                window = max(8, window // 2)
        return dict(op=op, B=B, N=N, S=S, Hq=g * Hkv, Hkv=Hkv, D=D, window=window, sinks=rng.choice([0, 1, 4, 16]))
    S = rng.choice([1, _log_int(rng, 1, 64), _log_int(rng, 1, 64)])
    S = max(1, min(S, 256 // g))
    cap = _log_int(rng, 1, 131072)
    B = max(1, min(_log_int(rng, 1, 64), (1 << 27) // (cap * Hkv * D), (1 << 28) // (cap * Hkv * g * S)))
    page = rng.choice([0, 16, 32, 64, 128])
    case = dict(op=op, B=B, S=S, Hq=g * Hkv, Hkv=Hkv, D=D, cap=cap, ragged=rng.random() < 0.7, page=page)
    if op == "window":
        case |= dict(window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 100]))
    if op == "mx":
        case |= dict(tree=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------ inputs --
def _lens(case):
    """Context lengths: all of the capacity, or spread over it (an empty one among eight or more)."""
    cap, B = case["cap"], case["B"]
    if not case["ragged"]:
        return [cap] * B
    lens = [1 + int(cap * ((n * 0.6180339887) % 1.0)) for n in range(B)]
    lens[0] = cap
    if B >= 8:
        lens[3] = 0
    return [min(x, cap) for x in lens]


def _normal(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * std).to(torch.bfloat16)


def _heavy_rows(gen, k):
    """One key row in a hundred four times as long: contexts hold a few tokens that many queries look at."""
    return k * (1 + 3 * (torch.rand(k.shape[:-1], generator=gen, device=DEV) < 0.01).to(k.dtype)).unsqueeze(-1)


def _parents(case, gen):
    """Drafted trees: node t hangs on the last committed token (-1) or on an earlier node; a sequence
    that drafted fewer tokens has absent nodes (-2) at its end, and one in eight drafted none."""
    B, S = case["B"], case["S"]
    t = torch.arange(S, device=DEV)
    far = torch.rand((B, S), generator=gen, device=DEV)
    par = torch.floor(t - 1 - (far ** 3) * t.clamp(max=4)).clamp(min=-1)
    count = torch.randint((S + 1) // 2, S + 1, (B,), generator=gen, device=DEV)
    if B >= 8:
        count[5] = 0
    return torch.where(t < count[:, None], par, torch.full_like(par, -2)).to(torch.int32).contiguous()


def _quantised(x):
    """[..., D] in e4m3 with one power-of-two scale per 32 elements (the exponent plus 127, in a byte):
    the smallest scale that keeps the block's largest magnitude within 448."""
    b = x.to(torch.float32).unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)                     # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)     # 448 = 0.875 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    q = torch.ldexp(torch.ldexp(b, (-e // 2).unsqueeze(-1)), (-e - (-e // 2)).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _values(q, scale):
    b = q.to(torch.float32).unflatten(-1, (-1, 32))
    e = scale.to(torch.int32) - 127
    half = torch.div(e, 2, rounding_mode="floor")
    return torch.ldexp(torch.ldexp(b, half.unsqueeze(-1)), (e - half).unsqueeze(-1)).flatten(-2)


def _paged(case, gen, *tensors):
    """The rows [B, Hkv, cap, ...] of each tensor in pages of a shuffled pool, and the page table."""
    B, P = case["B"], case["page"]
    per = -(-case["cap"] // P)
    table = torch.randperm(B * per + 3, generator=gen, device=DEV)[:B * per].reshape(B, per)
    pools = []
    for t in tensors:
        pad = torch.zeros(t.shape[:2] + (per * P,) + t.shape[3:], dtype=t.dtype, device=DEV)
        pad[:, :, :case["cap"]] = t
        rows = pad.unflatten(2, (per, P)).transpose(1, 2)            # [B, per, Hkv, P, ...]
        pool = torch.zeros((B * per + 3,) + rows.shape[2:], dtype=t.dtype, device=DEV)
        pool.view(torch.uint8)[table.flatten()] = rows.flatten(0, 1).contiguous().view(torch.uint8)
        pools.append(pool)
    return pools, table.to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    s = {"case": case}
    B = case["B"]
    if op == "train":
        N, Hq = case["N"], case["Hq"]
        s["q"], s["dout"] = (_normal(gen, (B, N, Hq, D)) for _ in range(2))
        s["k_ctx"], s["v_ctx"] = _heavy_rows(gen, _normal(gen, (B, Hkv, N, D))), _normal(gen, (B, Hkv, N, D))
        s["k_blk"], s["v_blk"] = (_normal(gen, (B, N, Hkv, D)) for _ in range(2))
        return s
    if op == "cache":
        T, cap = case["T"], case["cap"]
        s["k_new"], s["v_new"] = _heavy_rows(gen, _normal(gen, (B, T, Hkv, D))), _normal(gen, (B, T, Hkv, D))
        for x in "kv":
            s[x], s[x + "_scale"] = _quantised(_normal(gen, (B, Hkv, cap, D)))
            s[x + "_out"] = torch.zeros((B, Hkv, case["rows"], D), dtype=torch.bfloat16, device=DEV)
        held = torch.tensor([max(0, case["held"] - 3 * n) for n in range(B)], dtype=torch.int32, device=DEV)
        s["ctx_lens"], s["new_lens"] = held, held + T
        s["starts"] = (held + T - case["rows"]).clamp(min=0).to(torch.int32)
        return s
    S, Hq, cap = case["S"], case["Hq"], case["cap"]
    s["q"] = _normal(gen, (B, S, Hq, D))
    s["k_blk"], s["v_blk"] = (_normal(gen, (B, S, Hkv, D)) for _ in range(2))
    k, v = _heavy_rows(gen, _normal(gen, (B, Hkv, cap, D))), _normal(gen, (B, Hkv, cap, D))
    s["ctx_lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    s["table"] = None
    names = ["k_ctx", "v_ctx"]
    rows = [k, v]
    if op == "mx":
        names = ["k", "k_scale", "v", "v_scale"]
        rows = [*_quantised(k), *_quantised(v)]
    if case["page"]:
        rows, s["table"] = _paged(case, gen, *rows)
    s |= dict(zip(names, rows))
    s["parents"] = _parents(case, gen) if op == "tree" or case.get("tree") else None
    return s


# ------------------------------------------------------------- plain forms --
def _rows(x, Hkv):
    """[B, S, Hq, D] -> [B, Hkv, S*g, D] (row t*g + j), in 32 bits."""
    B, S, Hq, D = x.shape
    return x.to(torch.float32).unflatten(2, (Hkv, Hq // Hkv)).transpose(1, 2).reshape(B, Hkv, -1, D)


def _unrows(x, S):
    B, Hkv, R, D = x.shape
    return x.unflatten(2, (S, R // S)).transpose(1, 2).reshape(B, S, -1, D)


def _softmax_rows(q, k, v, visible, scale):
    """softmax(scale q k^T) v over the visible keys; rows that see none are 0."""
    s = torch.where(visible, scale * (q @ k.transpose(-1, -2)), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(l == 0, 1.0, l)


def _contiguous(pool, table, cap):
    """Pages [num, Hkv, P, ...] in table order -> [B, Hkv, cap, ...]."""
    if table is None:
        return pool
    return pool[table.long()].transpose(1, 2).flatten(2, 3)[:, :, :cap]


def _ancestors(parents):
    """[B, S, S]: whether row t sees block key u (u is t or an ancestor of it, and all of them are there)."""
    S = parents.shape[1]
    ids = torch.arange(S, device=parents.device)
    step = (parents.unsqueeze(-1) == ids).to(torch.float32)          # parent of t is u
    dead = (parents < -1).to(torch.float32)
    seen = torch.eye(S, device=parents.device).expand(parents.shape[0], S, S) + step
    # paths of up to 2, 4, 8, ... steps; 256 nodes need eight doublings
    twice = functools.reduce(lambda a, _: ((a @ a) > 0).to(torch.float32), range(8), seen)
    return (twice > 0) & ((twice @ dead.unsqueeze(-1)) == 0)


def _plain_decode(s, k_ctx, v_ctx):
    case = s["case"]
    B, S, Hkv, D, g = case["B"], case["S"], case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    L = s["ctx_lens"].long()[:, None]
    pos = torch.arange(k_ctx.shape[2], device=DEV)[None]
    if case["op"] == "window":
        # the positions that can be visible: the first tokens that lie before the window, and the window
        w, first = case["window"], torch.arange(case["sinks"], device=DEV)[None]
        last = L - w + torch.arange(w, device=DEV)[None]
        there = torch.cat([first < L - w, last >= 0], 1)
        at = torch.where(there, torch.cat([first.expand(B, -1), last], 1), 0)
        pick = at[:, None, :, None].expand(B, Hkv, -1, D)
        k_ctx, v_ctx = torch.gather(k_ctx, 2, pick), torch.gather(v_ctx, 2, pick)
    else:
        there = (pos < L).expand(B, -1)
    sees = there[:, None, :].expand(B, S, -1)
    block = torch.ones((B, S, S), dtype=torch.bool, device=DEV) if s["parents"] is None else _ancestors(s["parents"])
    alive = block.any(-1, keepdim=True)
    sees = torch.cat([sees & alive, block], -1).repeat_interleave(g, 1)[:, None]
    k = torch.cat([k_ctx, s["k_blk"].to(k_ctx.dtype).transpose(1, 2)], 2).to(torch.float32)
    v = torch.cat([v_ctx, s["v_blk"].to(v_ctx.dtype).transpose(1, 2)], 2).to(torch.float32)
    out = _softmax_rows(_rows(s["q"], Hkv), k, v, sees, 1 / math.sqrt(D))
    return _unrows(out, S).to(torch.bfloat16)


def _plain_train(s):
    case = s["case"]
    B, N, S, Hkv, D = case["B"], case["N"], case["S"], case["Hkv"], case["D"]
    NB, w, first = N // S, case["window"], torch.arange(case["sinks"], device=DEV)[None]
    start = S * torch.arange(NB, device=DEV)[:, None]
    last = start - w + torch.arange(w, device=DEV)[None]
    there = torch.cat([(first < start - w), last >= 0], 1)                       # [NB, sinks + w]
    at = torch.where(there, torch.cat([first.expand(NB, -1), last], 1), 0)

    def keys(ctx, blk):
        own_keys = blk.transpose(1, 2).unflatten(2, (NB, S))
        return torch.cat([ctx[:, :, at.flatten()].unflatten(2, at.shape), own_keys], 3).to(torch.float32)

    def rows(x):
        return _rows(x.unflatten(1, (NB, S)).flatten(0, 1), Hkv).unflatten(0, (B, NB)).transpose(1, 2)

    def unrows(x):
        return _unrows(x.transpose(1, 2).flatten(0, 1), S).unflatten(0, (B, NB)).flatten(1, 2).to(torch.bfloat16)

    def own_rows(x):
        return x.flatten(2, 3).transpose(1, 2).to(torch.bfloat16)

    sees = torch.cat([there, torch.ones((NB, S), dtype=torch.bool, device=DEV)], 1)[:, None]
    scale = 1 / math.sqrt(D)
    k, v, q, do = keys(s["k_ctx"], s["k_blk"]), keys(s["v_ctx"], s["v_blk"]), rows(s["q"]), rows(s["dout"])
    p = torch.where(sees, scale * (q @ k.transpose(-1, -2)), -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = p @ v
    ds = p * (do @ v.transpose(-1, -2) - (do * out).sum(-1, keepdim=True))
    dk = scale * (ds[..., -S:].transpose(-1, -2) @ q)
    dv = p[..., -S:].transpose(-1, -2) @ do
    return unrows(out), unrows(scale * (ds @ k)), own_rows(dk), own_rows(dv)


def _plain_cache(s):
    case = s["case"]
    B, T, cap, rows = case["B"], case["T"], case["cap"], case["rows"]
    n = torch.arange(B, device=DEV)[:, None]
    to = s["ctx_lens"].long()[:, None] + torch.arange(T, device=DEV)
    at = s["starts"].long()[:, None] + torch.arange(rows, device=DEV)
    there = (at < s["new_lens"].long()[:, None])[:, None, :, None]
    at = at.clamp(max=cap - 1)

    def pass_of(x):
        q, scale = _quantised(s[x + "_new"])
        s[x].view(torch.uint8)[n, :, to] = q.view(torch.uint8)
        s[x + "_scale"][n, :, to] = scale
        got = _values(s[x].view(torch.uint8)[n, :, at].view(torch.float8_e4m3fn), s[x + "_scale"][n, :, at])
        s[x + "_out"].copy_(torch.where(there, got.transpose(1, 2).to(torch.bfloat16), s[x + "_out"]))
        return s[x + "_out"]

    return pass_of("k"), pass_of("v")


# ------------------------------------------------------ the framework's calls --
@functools.lru_cache(maxsize=32)
def _plan(B, Hq, Hkv, D, S, cap=0, N=0, window=0, sinks=0, bf16=True):
    """The plan a program keeps for one shape."""
    from two_tower_block_b200 import ops
    return ops.Plan(B, Hq, Hkv, D, S, ctx_capacity=cap, seq_len=N, window=window, sinks=sinks, out_bf16=bf16)


def _own(s):
    from two_tower_block_b200 import ops
    case = s["case"]
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    if op == "train":
        plan = _plan(B, case["Hq"], Hkv, D, case["S"], N=case["N"], window=case["window"], sinks=case["sinks"],
                     bf16=False)
        x = s["q"], s["k_ctx"], s["v_ctx"], s["k_blk"], s["v_blk"]
        out, lse = plan.block_attn_block_causal(*x, want_lse=True)
        grads = plan.block_causal_backward(*x, out, lse, s["dout"])
        return tuple(t.to(torch.bfloat16) for t in (out, *grads))
    if op == "cache":
        plan = _plan(B, Hkv, Hkv, D, 1, cap=case["cap"])
        cache = ops.MxCache(s["k"], s["k_scale"], s["v"], s["v_scale"])
        plan.kv_append_mx(s["k_new"], s["v_new"], cache, s["ctx_lens"], advance=False)
        return plan.kv_read_mx(cache, s["new_lens"], s["starts"], s["k_out"], s["v_out"])
    plan = _plan(B, case["Hq"], Hkv, D, case["S"], cap=0 if case["page"] else case["cap"],
                 window=case.get("window", 0), sinks=case.get("sinks", 0))
    blk = s["k_blk"], s["v_blk"], s["ctx_lens"]
    if op == "mx":
        cache = ops.MxCache(s["k"], s["k_scale"], s["v"], s["v_scale"], page_table=s["table"])
        return plan.block_attn_mx(s["q"], cache, *blk, parents=s["parents"])
    if op == "tree":
        if case["page"]:
            return plan.block_attn_tree_paged(s["q"], s["k_ctx"], s["v_ctx"], s["table"], *blk, s["parents"])
        return plan.block_attn_tree(s["q"], s["k_ctx"], s["v_ctx"], *blk, s["parents"])
    if case["page"]:
        return plan.block_attn_paged(s["q"], s["k_ctx"], s["v_ctx"], s["table"], *blk)
    return plan.block_attn(s["q"], s["k_ctx"], s["v_ctx"], *blk)


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    if case["op"] == "train":
        return _plain_train(s)
    if case["op"] == "cache":
        return _plain_cache(s)
    if case["op"] == "mx":
        k, v = (_contiguous(s[x], s["table"], case["cap"]) for x in "kv")
        ks, vs = (_contiguous(s[x + "_scale"], s["table"], case["cap"]) for x in "kv")
        return _plain_decode(s, _values(k, ks), _values(v, vs))
    return _plain_decode(s, *(_contiguous(s[x], s["table"], case["cap"]) for x in ("k_ctx", "v_ctx")))


# ------------------------------------------------------------------- work --
def _visible(L, case):
    w = case.get("window", 0)
    return L if not w or L - w <= case["sinks"] else w + case["sinks"]


def work(case):
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    if op == "cache":
        new, back = B * case["T"] * Hkv * D * 2, 0
        for n in range(B):
            end = max(0, case["held"] - 3 * n) + case["T"]
            back += min(case["rows"], end) * Hkv * D * 2
        per = 1 + 1 / 32
        return {"bytes": new * (2 + per) + back * (2 + per), "flops": 3.0 * (new + back)}
    g, S = case["Hq"] // Hkv, case["S"]
    if op == "train":
        N = case["N"]
        ctx = sum(_visible(S * b, case) for b in range(N // S))
        pairs = B * case["Hq"] * S * (ctx + N)                # visible (row, key) pairs
        own_pairs = B * case["Hq"] * S * N
        rows, keys = B * N * case["Hq"] * D, B * N * Hkv * D
        # q, dout in; out, dq out; four key and value tensors in, two gradients out (2 bytes each)
        return {"bytes": 2.0 * (4 * rows + 6 * keys), "flops": 2.0 * D * (5 * pairs + 2 * own_pairs)}
    ctx = sum(_visible(L, case) for L in _lens(case))
    per = 1 + 1 / 32 if op == "mx" else 2
    io = 2 * B * S * case["Hq"] * D * 2 + 2 * B * S * Hkv * D * 2 + 4 * B
    if op == "tree" or case.get("tree"):
        io += 4 * B * S
    return {"bytes": io + 2 * ctx * Hkv * D * per, "flops": 4.0 * D * S * g * Hkv * (ctx + B * S)}


# ---------------------------------------------------------- 64-bit values --
def _exact_row_of(q, k, v, sees, scale):
    z = (q @ k.T) * scale
    z = z.masked_fill(~sees, -math.inf)
    top = z.max(dim=1).values
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(z - top[:, None])
    total = e.sum(1)
    return e, torch.where(total > 0, total, torch.ones_like(total)), z


def _exact_decode(case, s):
    B, S, Hq, Hkv, D, cap = (case[x] for x in ("B", "S", "Hq", "Hkv", "D", "cap"))
    g = Hq // Hkv
    out = torch.zeros((B, S, Hq, D), dtype=torch.float64, device=DEV)
    parents = s["parents"].tolist() if s["parents"] is not None else None

    def slab(name, n, h):
        if s["table"] is None:
            return s[name][n, h]
        return s[name][:, h][s["table"][n].long()].flatten(0, 1)[:cap]

    def decode8(name, n, h):
        q, e = slab(name, n, h), slab(name + "_scale", n, h).double() - 127
        return q.double() * torch.exp2(e).repeat_interleave(32, dim=1)

    for n, L in enumerate(_lens(case)):
        pos = torch.arange(cap, device=DEV)
        ctx = pos < L
        if case["op"] == "window":
            ctx &= (pos < case["sinks"]) | (pos >= L - case["window"])
        sees = torch.zeros((S, cap + S), dtype=torch.bool)
        for t in range(S):
            path, u = [], t
            if parents is None:
                path, u = list(range(S)), -1
            while u >= 0:
                path.append(u)
                u = parents[n][u]
            if u == -1:
                sees[t, :cap] = ctx.cpu()
                sees[t, [cap + x for x in path]] = True
        sees = sees.to(DEV).repeat_interleave(g, 0)
        for h in range(Hkv):
            if case["op"] == "mx":
                kc, vc = decode8("k", n, h), decode8("v", n, h)
            else:
                kc, vc = slab("k_ctx", n, h).double(), slab("v_ctx", n, h).double()
            k, v = torch.cat([kc, s["k_blk"][n, :, h].double()]), torch.cat([vc, s["v_blk"][n, :, h].double()])
            e, total, _ = _exact_row_of(s["q"][n, :, h * g:(h + 1) * g].reshape(S * g, D).double(), k, v, sees,
                                        D ** -0.5)
            out[n, :, h * g:(h + 1) * g] = ((e @ v) / total[:, None]).reshape(S, g, D)
    return out


def _exact_train(case, s):
    B, N, S, Hq, Hkv, D = (case[x] for x in ("B", "N", "S", "Hq", "Hkv", "D"))
    g, c = Hq // Hkv, D ** -0.5
    out, dq = (torch.zeros((B, N, Hq, D), dtype=torch.float64, device=DEV) for _ in range(2))
    dk, dv = (torch.zeros((B, N, Hkv, D), dtype=torch.float64, device=DEV) for _ in range(2))
    step = S * max(1, 1024 // S)
    pos = torch.arange(N, device=DEV)
    for n in range(B):
        for h in range(Hkv):
            kc, vc = s["k_ctx"][n, h].double(), s["v_ctx"][n, h].double()
            for a in range(0, N, step):
                b = min(N, a + step)
                hs = slice(h * g, (h + 1) * g)
                q, do = (s[x][n, a:b, hs].double().reshape(-1, D) for x in ("q", "dout"))
                kb, vb = (s[x][n, a:b, h].double() for x in ("k_blk", "v_blk"))
                start = (pos[a:b] // S * S)[:, None]
                ctx = (pos < start) & ((pos >= start - case["window"]) | (pos < case["sinks"]))
                sees = torch.cat([ctx, start == start.T], 1).repeat_interleave(g, 0)
                k, v = torch.cat([kc, kb]), torch.cat([vc, vb])
                e, total, _ = _exact_row_of(q, k, v, sees, c)
                p = e / total[:, None]
                o = p @ v
                ds = p * (do @ v.T - (do * o).sum(1)[:, None])
                out[n, a:b, hs] = o.reshape(b - a, g, D)
                dq[n, a:b, hs] = (c * (ds @ k)).reshape(b - a, g, D)
                dk[n, a:b, h] = c * (ds[:, N:].T @ q)
                dv[n, a:b, h] = p[:, N:].T @ do
    return out, dq, dk, dv


def _exact_cache(case, s):
    outs = []
    for x in "kv":
        new = s[x + "_new"].double().unflatten(-1, (-1, 32))
        amax = new.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)) / 448))
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
        e = torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e)
        e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)
        y = new * torch.exp2(-e)
        grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
        written = (torch.round(y / grid) * grid * torch.exp2(e)).flatten(-2).transpose(1, 2)
        held = s[x].double() * torch.exp2(s[x + "_scale"].double() - 127).repeat_interleave(32, dim=-1)
        back = s[x + "_out"].double()
        for n in range(case["B"]):
            L = int(s["ctx_lens"][n])
            held[n, :, L:L + case["T"]] = written[n]
            a = int(s["starts"][n])
            b = min(a + case["rows"], L + case["T"])
            back[n, :, :b - a] = held[n, :, a:b]
        outs.append(back)
    return tuple(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "train":
        return _exact_train(case, s)
    if case["op"] == "cache":
        return _exact_cache(case, s)
    return _exact_decode(case, s)
