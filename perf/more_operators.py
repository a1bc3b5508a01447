"""Cases that measure the operators of a speculative step whose drafted tokens form a tree.

Five operators over a paged KV pool [num_blocks][num_kv_heads][block_size][head_dim]. A sequence's context holds its
committed tokens and, behind them, the drafted ones of this step: nodes of a tree, parents before children.

  rope     queries and keys normed per head and rotated, queries out, keys and values into the pool
  layout   each node's mask of visible nodes (itself and its ancestors) and its position, from the parents
  tree     attention of the drafted tokens over the committed tokens and their own ancestors
  compact  K and V rows of the accepted path moved up behind the committed tokens, in every layer
  trim     the blocks behind the tokens that are kept, back onto the free stack

With ``own`` false, run() computes them from elementary torch operations in 32 bits; with ``own`` true it makes
the framework's calls. exact() is the definition again in 64 bits, sequence by sequence.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.bfloat16}  # of the queries and outputs
K_SCALE, V_SCALE = 0.015, 0.012  # of an 8-bit pool: near the largest value / 448


def listed():
    return [
        # two short chats, four drafted tokens each, four heads of 64: a call is all latency
        dict(name="tree-two-chats", op="tree", seqs=2, heads=4, kv_heads=4, dim=64, block=16, type="f16", ctx_lo=7,
             ctx_hi=33, q_lo=4, q_hi=4, softcap=0.0, window=0, roots=1),
        # a busy server's step of a grouped-query model: trees of up to 32 drafted tokens
        dict(name="tree-gqa-batch", op="tree", seqs=64, heads=32, kv_heads=8, dim=128, block=16, type="bf16",
             ctx_lo=128, ctx_hi=2048, q_lo=16, q_hi=32, softcap=0.0, window=0, roots=1),
        # an 8-bit cache, eight query heads to a kv head, capped scores, several drafts side by side
        dict(name="tree-e4m3-cap", op="tree", seqs=64, heads=64, kv_heads=8, dim=128, block=32, type="e4m3",
             ctx_lo=500, ctx_hi=4096, q_lo=8, q_hi=16, softcap=30.0, window=0, roots=3),
        # a few long contexts of a multi-head model: the whole cache is read
        dict(name="tree-mha-long", op="tree", seqs=4, heads=40, kv_heads=40, dim=128, block=16, type="f16",
             ctx_lo=9001, ctx_hi=32768, q_lo=17, q_hi=24, softcap=0.0, window=0, roots=1),
        # the drafted tokens of a step into an 8-bit pool
        dict(name="rope-step-e4m3", op="rope", tokens=256, heads=32, kv_heads=8, dim=128, block=16, type="e4m3",
             rotary=128, interleaved=False, norm=True, fused=True, pos_hi=8192, padding=0.1),
        # the prompts of a step, normed and rotated
        dict(name="rope-prompts", op="rope", tokens=16384, heads=32, kv_heads=8, dim=128, block=16, type="bf16",
             rotary=128, interleaved=False, norm=True, fused=True, pos_hi=131072, padding=0.0),
        # the trees of a small and of a full batch
        dict(name="layout-few", op="layout", seqs=8, ctx_lo=10, ctx_hi=500, q_lo=7, q_hi=16, roots=1),
        dict(name="layout-batch", op="layout", seqs=512, ctx_lo=1, ctx_hi=8192, q_lo=33, q_hi=64, roots=1),
        # one layer's accepted rows; those of all layers of a model at once
        dict(name="compact-layer", op="compact", seqs=64, layers=1, kv_heads=8, dim=128, block=16, type="bf16",
             ctx_lo=16, ctx_hi=512, q_lo=16, q_hi=32, roots=1),
        dict(name="compact-model", op="compact", seqs=128, layers=32, kv_heads=8, dim=128, block=16, type="e4m3",
             ctx_lo=16, ctx_hi=256, q_lo=33, q_hi=64, roots=1),
        # the drafted tokens that were not accepted give their blocks back
        dict(name="trim-step", op="trim", seqs=256, block=16, ctx_lo=1, ctx_hi=8192, drop=64),
        # most of a long rollout is taken back
        dict(name="trim-rewind", op="trim", seqs=4096, block=32, ctx_lo=0, ctx_hi=4096, drop=4096),
    ]


HEADS = [(8, 8), (40, 40), (32, 8), (64, 8), (16, 2), (12, 4), (16, 1), (20, 4)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "rope", "layout", "compact", "trim"])
    if op == "trim":
        hi = _log(rng, 16, 8192)
        return dict(op=op, seqs=_log(rng, 1, 4096), block=rng.choice([8, 16, 32]), ctx_lo=rng.randint(0, hi // 2),
                    ctx_hi=hi, drop=_log(rng, 1, hi))
    q_hi = _log(rng, 1, 256)
    trees = dict(q_lo=rng.randint(max(1, q_hi // 3), q_hi), q_hi=q_hi, roots=rng.choice([1, 1, 4]))
    if op == "layout":
        return dict(op=op, seqs=_log(rng, 1, min(1024, (1 << 22) // (q_hi * q_hi))), ctx_lo=0,
                    ctx_hi=_log(rng, 1, 32768), **trees)
    type_ = rng.choice(["f16", "bf16", "bf16", "e4m3"])
    heads, kv_heads = rng.choice(HEADS)
    dim = 128 if type_ == "e4m3" else rng.choice([64, 128])
    c = dict(op=op, kv_heads=kv_heads, dim=dim, block=rng.choice([8, 16, 32]), type=type_)
    if op == "rope":
        tokens = min(_log(rng, 1, 16384), 16384 * 48 // (heads + 2 * kv_heads))
        return dict(c, heads=heads, tokens=tokens, rotary=rng.choice([dim, dim, dim, dim // 2, dim // 4, 0]),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.6, fused=rng.random() < 0.5,
                    pos_hi=_log(rng, 64, 131072), padding=rng.choice([0.0, 0.1]))
    if op == "compact":
        ctx_hi = _log(rng, 16, 512)
        seqs = _log(rng, 1, 128)
        layers = min(_log(rng, 1, 48), max(1, (1 << 19) // (seqs * (ctx_hi + q_hi) * kv_heads // 16 + 1)))
        return dict(c, seqs=seqs, layers=layers, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, **trees)
    ctx_hi = _log(rng, 16, 32768)
    most = min(3_000_000 // (ctx_hi * kv_heads), 100_000_000 // (heads * q_hi * (ctx_hi + q_hi)))
    if most < 1:  # a long context: fewer drafted tokens
        q_hi = max(1, 100_000_000 // (heads * (ctx_hi + q_hi)))
        trees.update(q_lo=max(1, q_hi // 2), q_hi=q_hi)
    return dict(c, heads=heads, seqs=_log(rng, 1, max(1, min(128, most))), ctx_lo=rng.randint(ctx_hi // 4, ctx_hi),
                ctx_hi=ctx_hi, softcap=rng.choice([0.0, 0.0, 30.0]),
                window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), **trees)


def _random(c, what=""):
    return random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")) + what)


def _lengths(c):
    """Committed and drafted tokens of each sequence (trim: tokens, and tokens to keep). They are the case's own, so
    that work() knows them."""
    r = _random(c)
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    ctx[r.randrange(c["seqs"])] = c["ctx_hi"]
    if c["op"] == "trim":
        return ctx, [max(0, n - r.randint(0, c["drop"])) for n in ctx]
    return ctx, [r.randint(c["q_lo"], c["q_hi"]) for _ in ctx]


def _trees(c, qlen):
    """Each sequence's parents: -1 for its roots, else an earlier node (recent ones more often: branches grow deep)."""
    r = _random(c, "tree")
    return [[-1 if i < c["roots"] else max(r.randrange(i), r.randrange(i)) for i in range(q)] for q in qlen]


def _chain(parents, i):
    return [i] if parents[i] < 0 else _chain(parents, parents[i]) + [i]


def _accepted(c, qlen):
    """An accepted path of each sequence: a node and its ancestors, root first; now and then nothing."""
    r = _random(c, "accepted")
    return [[] if r.random() < 0.1 else _chain(p, r.randrange(q)) for p, q in zip(_trees(c, qlen), qlen)]


def _blocks_of(n, block):
    return -(-n // block)


def _words(q):
    return _blocks_of(max(q), 32)


def work(c):
    if c["op"] == "trim":
        ctx, keep = _lengths(c)
        gone = sum(_blocks_of(n, c["block"]) - _blocks_of(k, c["block"]) for n, k in zip(ctx, keep))
        return {"bytes": 12 * c["seqs"] + 8 + 8 * gone, "flops": 0}
    if c["op"] == "rope":
        T, H, Hkv, D, R = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rotary"]
        elem = 1 if c["type"] == "e4m3" else 2
        stored = sum(_stored(c))
        angles = len(set(_positions(c))) * R * 4
        return {"bytes": 2 * T * (H + 2 * Hkv) * D + 2 * T * H * D + 2 * stored * Hkv * D * elem + 12 * T + angles,
                "flops": T * (H + Hkv) * (3 * R + (4 * D if c["norm"] else 0))}
    ctx, qlen = _lengths(c)
    T = sum(qlen)
    if c["op"] == "layout":
        return {"bytes": 4 * T + 8 * c["seqs"] + 4 * T * _words(qlen) + 4 * T, "flops": 0}
    elem = 1 if c["type"] == "e4m3" else 2
    Hkv, D = c["kv_heads"], c["dim"]
    if c["op"] == "compact":
        paths = _accepted(c, qlen)
        moved = sum(u != i for p in paths for i, u in enumerate(p))
        return {"bytes": 4 * c["layers"] * moved * Hkv * D * elem + 4 * sum(map(len, paths)) + 12 * c["seqs"],
                "flops": 0}
    H, W = c["heads"], c["window"]
    keys = pairs = 0
    for n, q, parents in zip(ctx, qlen, _trees(c, qlen)):
        depth = [len(_chain(parents, i)) - 1 for i in range(q)]
        first = [max(0, n + d - W + 1) if W else 0 for d in depth]
        keys += max(0, n - min(first)) + q
        pairs += sum(max(0, n - f) + d + 1 for f, d in zip(first, depth))
    return {"bytes": 2 * keys * Hkv * D * elem + 4 * T * H * D + 4 * T * _words(qlen) + 4 * _blocks_of(keys, c["block"]),
            "flops": 4 * pairs * H * D}


def _stored(c):
    """Which tokens have a slot (the others are padding)."""
    r = _random(c, "padding")
    return [r.random() >= c["padding"] for _ in range(c["tokens"])]


def _positions(c):
    """Positions of prompts' tokens in a row, from random starts on."""
    r = _random(c, "positions")
    got = []
    while len(got) < c["tokens"]:
        n = min(c["tokens"] - len(got), r.randint(1, 1024), c["pos_hi"])
        start = r.randint(0, c["pos_hi"] - n)
        got += range(start, start + n)
    return got


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(ctx, block, g, spare):
    """Block tables over a shuffled pool, the blocks not used, and the number of blocks of the pool."""
    used = torch.tensor([_blocks_of(n, block) for n in ctx])
    num_blocks = int(used.sum()) + spare
    perm = torch.randperm(num_blocks, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    col = torch.arange(max(1, int(used.max())), device=DEV)
    at = ((torch.cumsum(used, 0) - used).to(DEV)[:, None] + col).clamp(max=num_blocks - 1)
    tables = torch.where(col < used.to(DEV)[:, None], perm[at], -1).to(torch.int32).contiguous()
    return tables, perm[int(used.sum()):].contiguous(), num_blocks


def _starts(qlen):
    return torch.tensor([0] + qlen, device=DEV).cumsum(0).to(torch.int32)


def _pools(c, shape, g):
    if c["type"] == "e4m3":  # codes as the quantizing write leaves them
        return [(torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).float() / s).clamp(-448, 448)
                .to(torch.float8_e4m3fn).view(torch.uint8) for s in (K_SCALE, V_SCALE)]
    return [torch.randn(shape, generator=g, device=DEV, dtype=TYPES[c["type"]]) for _ in range(2)]


def _angles(c):
    """The table of cosines and sines that a model keeps, [position][cos .. sin ..] in fp32, from 64 bits."""
    R = c["rotary"]
    if not R:
        return None
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
    a = torch.arange(c["pos_hi"], dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_rope(c, g):
    T, H, Hkv, D, B = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    dt = TYPES[c["type"]]
    num_blocks = _blocks_of(T, B) + 3
    slots = torch.randperm(num_blocks * B, generator=g, device=DEV)[:T]  # (ordinary steps fill blocks in a row; so
    if T > 64:  # do these: runs of slots from random blocks)
        blocks = torch.randperm(num_blocks, generator=g, device=DEV)
        slots = (blocks[:, None] * B + torch.arange(B, device=DEV)).reshape(-1)[:T].contiguous()
    slots = torch.where(torch.tensor(_stored(c), device=DEV), slots, -1)
    if c["fused"]:  # parts of one projection's output
        qkv = torch.randn((T, H + 2 * Hkv, D), generator=g, device=DEV).to(dt)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        q, k, v = (torch.randn((T, n, D), generator=g, device=DEV).to(dt) for n in (H, Hkv, Hkv))
    kc, vc = _pools(c, (num_blocks, Hkv, B, D), g)
    weights = [1.0 + 0.2 * torch.randn(D, generator=g, device=DEV) if c["norm"] else None for _ in range(2)]
    return dict(case=c, query=q, key=k, value=v, key_cache=kc, value_cache=vc, slots=slots,
                positions=_i32(_positions(c)) if c["rotary"] else None, cos_sin=_angles(c), q_weight=weights[0],
                k_weight=weights[1])


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] == "rope":
        return _prepare_rope(c, g)
    ctx, qlen = _lengths(c)
    if c["op"] == "trim":
        tables, free, num_blocks = _tables(ctx, c["block"], g, 7)
        stack = torch.full((num_blocks,), -1, dtype=torch.int32, device=DEV)
        stack[:free.numel()] = free
        return dict(case=c, block_tables=tables, context_lens=_i32(ctx), keep_lens=_i32(qlen), free_blocks=stack,
                    num_free=_i32([free.numel()]), num_blocks=num_blocks)
    st = dict(case=c, context_lens=_i32([n + q for n, q in zip(ctx, qlen)]), query_start_loc=_starts(qlen),
              max_q=max(qlen), rows=sum(qlen))
    if c["op"] == "layout":  # a random earlier node, or a root
        i = torch.cat([torch.arange(q, device=DEV) for q in qlen])
        u = torch.rand((2, st["rows"]), generator=g, device=DEV, dtype=torch.float64)
        up = (u * i).long().amax(0).minimum(i - 1)
        return dict(st, parents=torch.where(i < c["roots"], -1, up).to(torch.int32))
    H, Hkv, D, B = c.get("heads"), c["kv_heads"], c["dim"], c["block"]
    tables, _, num_blocks = _tables([n + q for n, q in zip(ctx, qlen)], B, g, 5)
    st["block_tables"] = tables
    if c["op"] == "compact":
        kc, vc = _pools(c, (c["layers"], num_blocks, Hkv, B, D), g)
        paths = _accepted(c, qlen)
        width = max(1, max(map(len, paths)))
        return dict(st, key_cache=kc, value_cache=vc, accepted=_i32([p + [-1] * (width - len(p)) for p in paths]),
                    num_accepted=_i32([len(p) for p in paths]))
    kc, vc = _pools(c, (num_blocks, Hkv, B, D), g)
    dt = TYPES[c["type"]]
    q = (torch.randn((st["rows"], H, D), generator=g, device=DEV) * 2.5).to(dt)  # scores with a spread of about 2.5
    W, masks, begin = _words(qlen), [], []
    for n, parents in zip(ctx, _trees(c, qlen)):
        bits = []
        for i, p in enumerate(parents):
            bits.append((1 << i) | (bits[p] if p >= 0 else 0))
            begin.append(max(0, n + bin(bits[-1]).count("1") - c["window"]))
        masks += [[(b >> (32 * w)) & 0xFFFFFFFF for w in range(W)] for b in bits]
    mask = torch.tensor(masks, dtype=torch.int64, device=DEV)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    return dict(st, query=q, key_cache=kc, value_cache=vc, tree_mask=mask, scale=D ** -0.5,
                max_ctx=max(n + q for n, q in zip(ctx, qlen)), key_begin=_i32(begin) if c["window"] else None)


# ---- the framework's calls


def _own(st):
    from paged_kv_cache_91_gb300 import binding as pkv

    c = st["case"]
    e4m3 = c.get("type") == "e4m3"
    if c["op"] == "rope":
        out = torch.empty(st["query"].shape, dtype=st["query"].dtype, device=DEV)
        args = [out, st["query"], st["key"], st["value"], st["key_cache"], st["value_cache"], st["slots"],
                st["positions"], st["cos_sin"]]
        kw = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6, interleaved=c["interleaved"])
        if e4m3:
            pkv.paged_kv_write_rope_fp8(*args, K_SCALE, V_SCALE, **kw)
        else:
            pkv.paged_kv_write_rope(*args, **kw)
        return dict(_stored_values(st), query=out)
    if c["op"] == "layout":
        mask = torch.empty((st["rows"], _blocks_of(st["max_q"], 32)), dtype=torch.int32, device=DEV)
        positions = torch.empty(st["rows"], dtype=torch.int32, device=DEV)
        pkv.paged_kv_tree_layout(st["parents"], st["query_start_loc"], st["context_lens"], mask, positions,
                                 max_query_len=st["max_q"])
        return {"mask": mask, "positions": positions}
    if c["op"] == "compact":
        pkv.paged_kv_compact_accepted(st["key_cache"], st["value_cache"], st["block_tables"], st["context_lens"],
                                      st["query_start_loc"], st["accepted"], st["num_accepted"])
        return _stored_values(st)
    if c["op"] == "trim":
        ctx_out, free_out = torch.empty_like(st["context_lens"]), torch.empty_like(st["num_free"])
        pkv.paged_kv_trim_blocks(st["block_tables"], st["context_lens"], st["keep_lens"], st["free_blocks"],
                                 st["num_free"], ctx_out, free_out, c["block"], st["num_blocks"])
        return {"free_blocks": st["free_blocks"], "context_lens": ctx_out, "num_free": free_out}
    out = torch.empty_like(st["query"])
    args = [out, st["query"], st["key_cache"], st["value_cache"], st["block_tables"], st["context_lens"],
            st["query_start_loc"], st["tree_mask"], st["scale"]]
    kw = dict(softcap=c["softcap"], key_begin=st["key_begin"], max_query_len=st["max_q"],
              max_context_len=st["max_ctx"])
    if e4m3:
        pkv.paged_attention_tree_fp8(*args, K_SCALE, V_SCALE, **kw)
    else:
        pkv.paged_attention_tree(*args, **kw)
    return out


def _stored_values(st):
    """The pools, 8-bit codes as the values (in units of the scale) that they stand for."""
    pools = {"key_cache": st["key_cache"], "value_cache": st["value_cache"]}
    if st["case"]["type"] == "e4m3":
        return {k: p.view(torch.float8_e4m3fn) for k, p in pools.items()}
    return pools


# ---- the plain forms


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight


def _rotated(x, st):
    c, R = st["case"], st["case"]["rotary"]
    if not R:
        return x
    angles = st["cos_sin"][st["positions"].long()][:, None]
    cos, sin = angles[..., :R // 2], angles[..., R // 2:]
    turn, rest = x[..., :R], x[..., R:]
    if c["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turn[..., :R // 2], turn[..., R // 2:]
        turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turn, rest], -1)


def _plain_rope(st):
    c, slots, B = st["case"], st["slots"], st["case"]["block"]
    q = _rotated(_normed(st["query"], st["q_weight"]), st).to(st["query"].dtype)
    k = _rotated(_normed(st["key"], st["k_weight"]), st)
    has = slots >= 0
    blk, off = slots[has] // B, slots[has] % B
    if c["type"] == "e4m3":
        for pool, x, scale in ((st["key_cache"], k, K_SCALE), (st["value_cache"], st["value"].float(), V_SCALE)):
            pool[blk, :, off] = (x[has] / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        st["key_cache"][blk, :, off] = k[has].to(st["key_cache"].dtype)
        st["value_cache"][blk, :, off] = st["value"][has]
    return dict(_stored_values(st), query=q)


def _plain_layout(st):
    """Reachability by squaring the matrix of parents, every sequence padded to the longest."""
    starts, ctx, Q = st["query_start_loc"].long(), st["context_lens"].long(), st["max_q"]
    qlen = starts[1:] - starts[:-1]
    i = torch.arange(Q, device=DEV)
    real = i < qlen[:, None]
    row = (starts[:-1, None] + i).clamp(max=st["rows"] - 1)
    parent = torch.where(real, st["parents"].long()[row], -1)
    see = ((parent[:, :, None] == i) | (i[:, None] == i)).float()  # [S][node][itself or its parent]
    for _ in range(max(1, math.ceil(math.log2(Q)))) if Q > 1 else ():
        see = (see @ see).clamp(max=1.0)
    W = _blocks_of(Q, 32)
    bits = torch.nn.functional.pad(see.long(), (0, 32 * W - Q)).view(-1, Q, W, 32)
    mask = (bits << torch.arange(32, device=DEV)).sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    positions = (ctx - qlen)[:, None] + see.sum(-1).long() - 1
    return {"mask": mask[real], "positions": positions[real].to(torch.int32)}


def _gather(pool, scale, blk, off, c):
    x = pool[blk, :, off]  # [S][L][Hkv][D]
    return x.view(torch.float8_e4m3fn).float() * scale if c["type"] == "e4m3" else x.float()


def _plain_tree(st):
    """Every sequence's rows side by side (padded to the longest), over its context."""
    c = st["case"]
    H, Hkv, D, B = c["heads"], c["kv_heads"], c["dim"], c["block"]
    ctx, starts = st["context_lens"].long(), st["query_start_loc"].long()
    S, Q, G, L = ctx.numel(), st["max_q"], H // Hkv, st["max_ctx"]
    qlen = starts[1:] - starts[:-1]
    i = torch.arange(Q, device=DEV)
    row = (starts[:-1, None] + i).clamp(max=st["rows"] - 1)  # [S][Q]
    real = i < qlen[:, None]
    j = torch.arange(L, device=DEV)
    node = j - (ctx - qlen)[:, None]  # [S][L]: the drafted token of a key, below 0 a committed one
    words = st["tree_mask"][row]  # [S][Q][W]
    word = (node >> 5).clamp(0, words.shape[2] - 1)[:, None].expand(S, Q, L)
    see = (node[:, None] < 0) | (((words.gather(2, word) >> (node & 31)[:, None].int()) & 1) != 0)
    see &= (j < ctx[:, None])[:, None]
    if st["key_begin"] is not None:
        see &= j >= st["key_begin"].long()[row][..., None]
    blk = st["block_tables"].gather(1, (j // B).expand(S, L)).long().clamp(min=0)
    k = _gather(st["key_cache"], K_SCALE, blk, (j % B).expand(S, L), c)
    q = st["query"][row].float().view(S, Q, Hkv, G, D)
    x = torch.einsum("sqhgd,slhd->shgql", q, k).mul_(st["scale"])  # [S][Hkv][G][Q][L]
    del k
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    x.masked_fill_(~see[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == float("-inf"), 0.0, m)).exp_()
    l = x.sum(-1)  # [S][Hkv][G][Q]
    v = _gather(st["value_cache"], V_SCALE, blk, (j % B).expand(S, L), c)
    o = torch.einsum("shgql,slhd->sqhgd", x, v)
    o = o / torch.where(l > 0, l, 1.0).permute(0, 3, 1, 2)[..., None]
    out = torch.empty_like(st["query"])
    out[row[real]] = o.reshape(S, Q, H, D)[real].to(out.dtype)
    return out


def _plain_compact(st):
    B, acc = st["case"]["block"], st["accepted"].long()
    starts, ctx, tables = st["query_start_loc"].long(), st["context_lens"].long(), st["block_tables"].long()
    first = ctx - (starts[1:] - starts[:-1])
    i = torch.arange(acc.shape[1], device=DEV)
    s, i = ((i < st["num_accepted"].long()[:, None]) & (acc != i)).nonzero(as_tuple=True)
    src, dst = first[s] + acc[s, i], first[s] + i
    sb, so, db, do = tables[s, src // B], src % B, tables[s, dst // B], dst % B
    st["key_cache"][:, db, :, do] = st["key_cache"][:, sb, :, so]  # (the right side is gathered first)
    st["value_cache"][:, db, :, do] = st["value_cache"][:, sb, :, so]
    return _stored_values(st)


def _plain_trim(st):
    B = st["case"]["block"]
    ctx, keep, free = st["context_lens"].long(), st["keep_lens"].long(), st["num_free"].long()
    tables, stack = st["block_tables"], st["free_blocks"]
    have, held = (ctx + B - 1) // B, (keep + B - 1) // B
    count = have - held
    col = torch.arange(tables.shape[1], device=DEV)
    mine = (col >= held[:, None]) & (col < have[:, None])
    at = free + (torch.cumsum(count, 0) - have)[:, None] + col
    stack[at[mine]] = tables[mine]
    return {"free_blocks": stack, "context_lens": keep.to(torch.int32), "num_free": (free + count.sum()).to(torch.int32)}


PLAIN = {"rope": _plain_rope, "layout": _plain_layout, "tree": _plain_tree, "compact": _plain_compact,
         "trim": _plain_trim}


def run(st):
    if own:
        return _own(st)
    return PLAIN[st["case"]["op"]](st)


# ---- the definition in 64 bits


def _exact_rope(c, st):
    T, D, R, B = c["tokens"], c["dim"], c["rotary"], c["block"]
    got = {}
    for name, w in (("query", "q_weight"), ("key", "k_weight")):
        x = st[name].double()
        if c["norm"]:
            x = x / (x.square().sum(-1, keepdim=True) / D + 1e-6).sqrt() * st[w].double()
        if R:  # a pair is a complex number; its turn is a product with cos + i sin
            z = torch.complex(*(st["cos_sin"][st["positions"].long()].double().view(T, 1, 2, R // 2).unbind(2)))
            lo, hi = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
            z = z * torch.complex(x[..., lo], x[..., hi])
            x[..., lo], x[..., hi] = z.real, z.imag
        got[name] = x
    out = {"query": got["query"]}
    has = st["slots"] >= 0
    at = st["slots"][has]
    for name, x, scale in (("key_cache", got["key"], K_SCALE), ("value_cache", st["value"].double(), V_SCALE)):
        pool = st[name]
        if c["type"] == "e4m3":
            pool, x = pool.view(torch.float8_e4m3fn), (x / scale).clamp(-448, 448)
        pool = pool.double().transpose(1, 2).contiguous().view(-1, c["kv_heads"], D)  # [slot][head][D]
        pool[at] = x[has]
        out[name] = pool.view(-1, B, c["kv_heads"], D).transpose(1, 2).contiguous()
    return out


def exact(c, seed):
    if c["op"] in ("layout", "trim"):
        return None  # whole numbers
    st = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, st)
    B = c["block"]
    ctx, qlen = _lengths(c)
    if c["op"] == "compact":
        tables = st["block_tables"].tolist()
        for s, path in enumerate(_accepted(c, qlen)):
            for i, u in enumerate(path):  # root first: a row is read before it is overwritten
                (db, do), (sb, so) = ((tables[s][p // B], p % B) for p in (ctx[s] + i, ctx[s] + u))
                for pool in (st["key_cache"], st["value_cache"]):
                    pool[:, db, :, do] = pool[:, sb, :, so].clone()
        return _stored_values(st)
    H, Hkv, D = c["heads"], c["kv_heads"], c["dim"]
    G = H // Hkv
    out = torch.zeros(sum(qlen), H, D, dtype=torch.float64, device=DEV)
    at = 0
    for s, (n, q, parents) in enumerate(zip(ctx, qlen, _trees(c, qlen))):
        see = torch.zeros(q, n + q, dtype=torch.bool)
        for i in range(q):
            chain = _chain(parents, i)
            first = max(0, n + len(chain) - c["window"]) if c["window"] else 0
            see[i, :n] = True
            see[i, [n + u for u in chain]] = True
            see[i, :first] = False
        see = see.to(DEV)
        blocks = st["block_tables"][s, :_blocks_of(n + q, B)].long()
        for h in range(Hkv):
            kv = []
            for pool, scale in ((st["key_cache"], K_SCALE), (st["value_cache"], V_SCALE)):
                x = pool[blocks, h].reshape(-1, D)[:n + q]
                kv.append(x.view(torch.float8_e4m3fn).double() * scale if c["type"] == "e4m3" else x.double())
            for g in range(G):
                x = st["query"][at:at + q, h * G + g].double() @ kv[0].T * st["scale"]
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                w = torch.softmax(x.masked_fill(~see, float("-inf")), -1)
                out[at:at + q, h * G + g] = torch.where(see.any(-1, keepdim=True), w, 0.0) @ kv[1]
        at += q
    return out
