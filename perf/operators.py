"""Cases that measure the scored paged attention and the block-table operators.

Four operators over a paged KV pool [num_blocks][num_kv_heads][block_size][head_dim]:

  decode   one query token per sequence; scores capped by a tanh, biased by distance, within a window or from a
           given first key on
  prompt   several query tokens per sequence (chunks, whole prompts, verified drafts), the same scores, and a
           visible key interval per query token (document masks, prefix masks)
  reserve  block tables, slot map and query offsets of the next step, from the request lengths
  release  the blocks of finished sequences back onto the free stack

With ``own`` false, run() computes them from elementary torch operations in 32 bits; with ``own`` true it makes
the framework's calls. exact() is the definition again in 64 bits, sequence by sequence.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.bfloat16}  # of the queries and outputs


def _decode(name, **kw):
    return dict(name=name, op="decode", q_lo=1, q_hi=1, whole=False, mask="causal", **kw)


def listed():
    return [
        # two short chats, four heads of 64: a call is all latency
        _decode("decode-two-short", seqs=2, heads=4, kv_heads=4, dim=64, block=16, type="f16", ctx_lo=7, ctx_hi=33,
                softcap=30.0, alibi=True, window=0),
        # a busy server's step of a grouped-query model whose layers cap their scores and see a window
        _decode("decode-gqa-cap-window", seqs=256, heads=32, kv_heads=8, dim=128, block=16, type="bf16", ctx_lo=64,
                ctx_hi=8192, softcap=50.0, alibi=False, window=1024),
        # a few long contexts of a multi-head model with distance biases: the whole cache is read
        _decode("decode-mha-long-alibi", seqs=12, heads=40, kv_heads=40, dim=128, block=16, type="f16", ctx_lo=9001,
                ctx_hi=16384, softcap=0.0, alibi=True, window=0),
        # an 8-bit cache, eight query heads to a kv head, each sequence attending from its own document on
        dict(_decode("decode-e4m3-cap-document", seqs=128, heads=64, kv_heads=8, dim=128, block=32, type="e4m3",
                     ctx_lo=500, ctx_hi=4096, softcap=30.0, alibi=False, window=0), mask="documents"),
        # a speculative step: four drafted tokens of each sequence are verified
        dict(name="prompt-verify-alibi", op="prompt", seqs=64, heads=40, kv_heads=40, dim=128, block=16, type="f16",
             ctx_lo=100, ctx_hi=512, q_lo=4, q_hi=4, whole=False, mask="causal", softcap=0.0, alibi=True, window=0),
        # ragged prefill chunks batched with decode tokens, capped scores within a window
        dict(name="prompt-chunks-cap-window", op="prompt", seqs=32, heads=32, kv_heads=8, dim=128, block=16,
             type="bf16", ctx_lo=300, ctx_hi=4096, q_lo=1, q_hi=128, whole=False, mask="causal", softcap=50.0,
             alibi=False, window=1024),
        # one long row of packed documents, as a batch of prompts that were joined into one
        dict(name="prompt-documents-cap", op="prompt", seqs=1, heads=32, kv_heads=8, dim=128, block=16, type="bf16",
             ctx_lo=16384, ctx_hi=16384, q_lo=0, q_hi=0, whole=True, mask="documents", softcap=50.0, alibi=False,
             window=0),
        # prompts over an 8-bit cache whose first part every token sees (a prefix mask), with distance biases
        dict(name="prompt-e4m3-prefix-alibi", op="prompt", seqs=8, heads=64, kv_heads=8, dim=128, block=16,
             type="e4m3", ctx_lo=700, ctx_hi=2048, q_lo=200, q_hi=512, whole=False, mask="prefix", softcap=0.0,
             alibi=True, window=0),
        # the next decode step's slots of a full batch
        dict(name="reserve-decode-step", op="reserve", seqs=256, block=16, ctx_lo=1, ctx_hi=8192, new_lo=1, new_hi=1,
             spare=64),
        # the slots of a step that admits long prompts next to decode tokens
        dict(name="reserve-long-prompts", op="reserve", seqs=1024, block=16, ctx_lo=0, ctx_hi=4096, new_lo=1,
             new_hi=511, spare=1000),
        # a step that finishes some of its sequences
        dict(name="release-step", op="release", seqs=256, block=16, ctx_lo=1, ctx_hi=8192, share=0.25),
        # a drained server gives back everything
        dict(name="release-everything", op="release", seqs=4096, block=32, ctx_lo=0, ctx_hi=4096, share=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prompt", "decode", "prompt", "reserve", "release"])
    if op in ("reserve", "release"):
        seqs, block = _log(rng, 1, 4096), rng.choice([8, 16, 32])
        hi = _log(rng, 16, 4096)
        c = dict(op=op, seqs=seqs, block=block, ctx_lo=rng.randint(0, hi // 2), ctx_hi=hi)
        if op == "release":
            return dict(c, share=rng.choice([0.05, 0.3, 0.7, 1.0]))
        new_hi = _log(rng, 1, max(1, min(2048, 262144 // seqs)))
        # a pool that runs out part of the way (spare < 0) leaves later sequences without
        return dict(c, new_lo=rng.randint(0, new_hi), new_hi=new_hi, spare=rng.choice([0, 3, 500, -20]))
    type_ = rng.choice(["f16", "bf16", "bf16", "e4m3"])
    heads, kv_heads = rng.choice([(8, 8), (40, 40), (32, 8), (64, 8), (16, 2), (12, 4), (16, 1), (20, 4)])
    dim = 128 if type_ == "e4m3" else rng.choice([64, 128])
    c = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, block=rng.choice([8, 16, 32]), type=type_,
             softcap=rng.choice([0.0, 20.0, 30.0, 50.0]), alibi=rng.random() < 0.4,
             window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    ctx_hi = _log(rng, 16, 16384 if op == "decode" else 4096)
    c.update(ctx_lo=rng.randint(1, ctx_hi), ctx_hi=ctx_hi)
    if op == "decode":
        return dict(c, seqs=max(1, min(_log(rng, 1, 256), 4_000_000 // (ctx_hi * kv_heads))), q_lo=1, q_hi=1,
                    whole=False, mask=rng.choice(["causal", "documents"]))
    seqs = max(1, min(_log(rng, 1, 64), 32768 // ctx_hi))
    whole = rng.random() < 0.3
    if whole:
        seqs = min(seqs, max(1, 4096 // ctx_hi))
    q_hi = min(ctx_hi, _log(rng, 1, 512))
    return dict(c, seqs=seqs, q_lo=0 if whole else rng.randint(1, min(q_hi, c["ctx_lo"])), q_hi=0 if whole else q_hi,
                whole=whole, mask=rng.choice(["causal", "documents", "prefix"]))


def _lengths(c):
    """The sequences' context lengths and query lengths. They are the case's own, so that work() knows them."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    ctx[r.randrange(c["seqs"])] = c["ctx_hi"]
    if c["op"] == "reserve":
        return ctx, [r.randint(c["new_lo"], c["new_hi"]) for _ in ctx]
    if c["op"] == "release":
        return ctx, [int(r.random() < c["share"]) for _ in ctx]
    if c["whole"]:
        return ctx, list(ctx)
    return ctx, [min(n, r.randint(c["q_lo"], c["q_hi"])) for n in ctx]


def _intervals(c, ctx, qlen):
    """Per query token the first visible key and the end of the visible keys, as the mask gives them."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")) + "mask")
    begin, end = [], []
    for n, q in zip(ctx, qlen):
        if c["mask"] == "documents" and c["op"] == "decode":
            begin.append(r.randint(0, n // 2))
        elif c["mask"] == "documents":
            start, left, at = 0, 0, []
            for j in range(n):
                if left == 0:
                    start, left = j, r.randint(max(1, n // 12), max(1, n // 3))
                left -= 1
                at.append(start)
            begin += at[n - q:]
        elif c["mask"] == "prefix":
            prefix = r.randint(0, n)
            end += [max(n - q + i + 1, prefix) for i in range(q)]
    return begin or None, end or None


def _blocks_of(n, block):
    return -(-n // block)


def _rows(c):
    """Per query token (first visible key, end of the visible keys) with the window, for work()."""
    ctx, qlen = _lengths(c)
    begin, end = _intervals(c, ctx, qlen)
    at, rows = 0, []
    for s, (n, q) in enumerate(zip(ctx, qlen)):
        for i in range(q):
            p = n - q + i
            lo = max(begin[at] if begin else 0, p - c["window"] + 1 if c["window"] else 0)
            rows.append((s, lo, max(lo, end[at] if end else p + 1)))
            at += 1
    return rows


def work(c):
    if c["op"] in ("reserve", "release"):
        ctx, new = _lengths(c)
        B = c["block"]
        if c["op"] == "release":
            gone = sum(_blocks_of(n, B) for n, f in zip(ctx, new) if f)
            return {"bytes": 12 * c["seqs"] + 8 + 8 * gone, "flops": 0}
        fresh = sum(_blocks_of(n + k, B) - _blocks_of(n, B) for n, k in zip(ctx, new))
        return {"bytes": 20 * c["seqs"] + 12 + 8 * fresh + 8 * sum(new), "flops": 0}
    rows = _rows(c)
    elem, H, Hkv, D = (1 if c["type"] == "e4m3" else 2), c["heads"], c["kv_heads"], c["dim"]
    lo, hi = {}, {}
    for s, a, b in rows:
        if b > a:
            lo[s], hi[s] = min(lo.get(s, a), a), max(hi.get(s, b), b)
    keys = sum(hi[s] - lo[s] for s in lo)
    pairs = sum(b - a for _, a, b in rows)
    return {"bytes": 2 * keys * Hkv * D * elem + 4 * len(rows) * H * D + 4 * _blocks_of(keys, c["block"]),
            "flops": 4 * pairs * H * D}


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(ctx, extra, block, g, spare):
    """Block tables over a shuffled pool with room for `extra` more tokens each; the blocks not yet used, and
    the number of blocks of the pool."""
    used = torch.tensor([_blocks_of(n, block) for n in ctx])
    full = torch.tensor([max(1, _blocks_of(n + k, block)) for n, k in zip(ctx, extra)])
    fresh = int((full - used).clamp(min=0).sum())
    num_blocks = int(used.sum()) + max(1, fresh + spare)
    perm = torch.randperm(num_blocks, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = int(full.max())
    first = (torch.cumsum(used, 0) - used).to(DEV)
    col = torch.arange(width, device=DEV)
    at = (first[:, None] + col).clamp(max=num_blocks - 1)
    tables = torch.where(col < used.to(DEV)[:, None], perm[at], -1).to(torch.int32).contiguous()
    return tables, perm[int(used.sum()):].contiguous(), num_blocks


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ctx, new = _lengths(c)
    st = {"case": c, "context_lens": _i32(ctx)}
    if c["op"] == "release":
        tables, free, num_blocks = _tables(ctx, [0] * len(ctx), c["block"], g, 7)
        stack = torch.full((num_blocks,), -1, dtype=torch.int32, device=DEV)
        stack[:free.numel()] = free
        return dict(st, block_tables=tables, free_blocks=stack, num_free=_i32([free.numel()]), finished=_i32(new),
                    num_blocks=num_blocks)
    if c["op"] == "reserve":
        tables, free, num_blocks = _tables(ctx, new, c["block"], g, c["spare"])
        return dict(st, block_tables=tables, free_blocks=free, num_free=_i32([free.numel()]), new_lens=_i32(new),
                    tokens=sum(new) + 13, num_blocks=num_blocks)
    H, Hkv, D, B = c["heads"], c["kv_heads"], c["dim"], c["block"]
    dt = TYPES[c["type"]]
    tables, _, num_blocks = _tables(ctx, [0] * len(ctx), B, g, 5)
    shape = (num_blocks, Hkv, B, D)
    if c["type"] == "e4m3":  # codes as the quantizing write leaves them: values over a scale near their maximum / 448
        st.update(k_scale=0.015, v_scale=0.012)
        pools = []
        for scale in (0.015, 0.012):
            x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).float() / scale
            pools.append(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        pools = [torch.randn(shape, generator=g, device=DEV, dtype=dt) for _ in range(2)]
    rows = sum(new)
    q = (torch.randn((rows, H, D), generator=g, device=DEV) * 2.5).to(dt)  # scores with a spread of about 2.5
    begin, end = _intervals(c, ctx, new)
    starts = [0]
    for k in new:
        starts.append(starts[-1] + k)
    return dict(st, query=q, key_cache=pools[0], value_cache=pools[1], block_tables=tables,
                query_start_loc=_i32(starts), scale=D ** -0.5, max_ctx=max(ctx), max_q=max(new),
                slopes=torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)
                if c["alibi"] else None,
                key_begin=_i32(begin) if begin else None, key_end=_i32(end) if end else None)


# ---- the framework's calls


def _own(st):
    from paged_kv_cache_91_gb300 import binding as pkv

    c = st["case"]
    if c["op"] == "release":
        ctx_out, free_out = torch.empty_like(st["context_lens"]), torch.empty_like(st["num_free"])
        pkv.paged_kv_release_blocks(st["block_tables"], st["context_lens"], st["finished"], st["free_blocks"],
                                    st["num_free"], ctx_out, free_out, c["block"], st["num_blocks"])
        return {"free_blocks": st["free_blocks"], "context_lens": ctx_out, "num_free": free_out}
    if c["op"] == "reserve":
        S = st["context_lens"].numel()
        slots = torch.empty(st["tokens"], dtype=torch.int64, device=DEV)
        starts = torch.empty(S + 1, dtype=torch.int32, device=DEV)
        ctx_out, granted = torch.empty_like(st["context_lens"]), torch.empty_like(st["context_lens"])
        free_out = torch.empty_like(st["num_free"])
        pkv.paged_kv_reserve_slots(st["block_tables"], st["context_lens"], st["new_lens"], st["free_blocks"],
                                   st["num_free"], slots, starts, ctx_out, free_out, granted, c["block"],
                                   st["num_blocks"])
        return {"block_tables": st["block_tables"], "slots": slots, "starts": starts, "context_lens": ctx_out,
                "granted": granted, "num_free": free_out}
    out = torch.empty_like(st["query"])
    args = [out, st["query"], st["key_cache"], st["value_cache"], st["block_tables"], st["context_lens"]]
    kw = dict(softcap=c["softcap"], alibi_slopes=st["slopes"], window=c["window"], key_begin=st["key_begin"],
              max_context_len=st["max_ctx"])
    if c["type"] == "e4m3":
        kw.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
    if c["op"] == "prompt":
        call = (pkv.paged_attention_multi_query_scored_fp8 if c["type"] == "e4m3"
                else pkv.paged_attention_multi_query_scored)
        call(*args, st["query_start_loc"], st["scale"], key_end=st["key_end"], max_query_len=st["max_q"], **kw)
    else:
        call = pkv.paged_attention_decode_scored_fp8 if c["type"] == "e4m3" else pkv.paged_attention_decode_scored
        call(*args, st["scale"], **kw)
    return out


# ---- the plain forms


def _gather(pool, scale, blk, off, c):
    x = pool[blk, :, off]  # [S][L][Hkv][D]
    return x.view(torch.float8_e4m3fn).float() * scale if c["type"] == "e4m3" else x.float()


def _plain_attention(st):
    """Every sequence's rows side by side (padded to the longest), over the keys that some row may see."""
    c = st["case"]
    H, Hkv, D, B, W = c["heads"], c["kv_heads"], c["dim"], c["block"], c["window"]
    ctx, starts = st["context_lens"].long(), st["query_start_loc"].long()
    S, Q, G = ctx.numel(), st["max_q"], H // Hkv
    qlen = starts[1:] - starts[:-1]
    first = ctx - qlen  # position of the first query token
    i = torch.arange(Q, device=DEV)
    row = (starts[:-1, None] + i).clamp(max=st["query"].shape[0] - 1)  # [S][Q]
    real = i < qlen[:, None]
    p = first[:, None] + i
    L = min(st["max_ctx"], W + Q - 1) if W else st["max_ctx"]
    base = (first - W + 1).clamp(min=0) if W else torch.zeros_like(first)
    j = base[:, None] + torch.arange(L, device=DEV)  # [S][L] key positions
    lo = st["key_begin"].long()[row] if st["key_begin"] is not None else torch.zeros_like(p)
    hi = st["key_end"].long()[row] if st["key_end"] is not None else p + 1
    if W:
        lo = torch.maximum(lo, p - W + 1)
    hi = torch.minimum(hi, ctx[:, None])
    see = (j[:, None] >= lo[:, :, None]) & (j[:, None] < hi[:, :, None])  # [S][Q][L]
    blk = st["block_tables"].gather(1, (j // B).clamp(max=st["block_tables"].shape[1] - 1)).long().clamp(min=0)
    k = _gather(st["key_cache"], st.get("k_scale"), blk, j % B, c)
    q = st["query"][row].float().view(S, Q, Hkv, G, D)
    x = torch.einsum("sqhgd,slhd->shgql", q, k).mul_(st["scale"])  # [S][Hkv][G][Q][L]
    del k
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if st["slopes"] is not None:
        far = (p[:, :, None] - j[:, None]).abs().float()
        x -= st["slopes"].view(1, Hkv, G, 1, 1) * far[:, None, None]
    x.masked_fill_(~see[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == float("-inf"), 0.0, m)).exp_()
    l = x.sum(-1)  # [S][Hkv][G][Q]
    v = _gather(st["value_cache"], st.get("v_scale"), blk, j % B, c)
    o = torch.einsum("shgql,slhd->sqhgd", x, v)
    o = o / torch.where(l > 0, l, 1.0).permute(0, 3, 1, 2)[..., None]
    out = torch.empty_like(st["query"])
    out[row[real]] = o.reshape(S, Q, H, D)[real].to(out.dtype)
    return out


def _plain_reserve(st):
    B, F = st["case"]["block"], st["free_blocks"]
    ctx, new, free = st["context_lens"].long(), st["new_lens"].long(), st["num_free"].long()
    tables, T = st["block_tables"], st["tokens"]
    have = (ctx + B - 1) // B
    need = (ctx + new + B - 1) // B - have
    taken = torch.cumsum(need, 0)
    granted = (need == 0) | (taken <= free)
    starts = torch.cat([torch.zeros_like(free), torch.cumsum(new, 0)])
    t = torch.arange(T, device=DEV)
    s = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=ctx.numel() - 1)
    pos = ctx[s] + t - starts[s]
    ok = (t < starts[-1]) & granted[s]
    col = pos // B
    fresh = col >= have[s]
    nth = (taken - need)[s] + col - have[s]
    phys = torch.where(fresh, F[(free - 1 - nth).clamp(0, F.numel() - 1)].long(),
                       tables[s, col.clamp(max=tables.shape[1] - 1)].long())
    slots = torch.where(ok, phys * B + pos % B, -1)
    first = ok & fresh & (pos % B == 0)
    tables[s[first], col[first]] = phys[first].to(torch.int32)
    return {"block_tables": tables, "slots": slots, "starts": starts.to(torch.int32),
            "context_lens": torch.where(granted, ctx + new, ctx).to(torch.int32),
            "granted": granted.to(torch.int32),
            "num_free": (free - (need * granted).sum()).to(torch.int32)}


def _plain_release(st):
    B = st["case"]["block"]
    ctx, gone, free = st["context_lens"].long(), st["finished"] != 0, st["num_free"].long()
    tables, stack = st["block_tables"], st["free_blocks"]
    count = torch.where(gone, (ctx + B - 1) // B, 0)
    col = torch.arange(tables.shape[1], device=DEV)
    mine = col < count[:, None]
    at = free + (torch.cumsum(count, 0) - count)[:, None] + col
    stack[at[mine]] = tables[mine]
    return {"free_blocks": stack, "context_lens": torch.where(gone, 0, ctx).to(torch.int32),
            "num_free": (free + count.sum()).to(torch.int32)}


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    return _plain_reserve(st) if op == "reserve" else _plain_release(st) if op == "release" else _plain_attention(st)


# ---- the definition in 64 bits


def exact(c, seed):
    if c["op"] in ("reserve", "release"):
        return None  # whole numbers
    st = prepare(c, seed)
    ctx, qlen = _lengths(c)
    begin, end = _intervals(c, ctx, qlen)
    H, Hkv, D, B, W = c["heads"], c["kv_heads"], c["dim"], c["block"], c["window"]
    G = H // Hkv
    out = torch.zeros(sum(qlen), H, D, dtype=torch.float64, device=DEV)
    at = 0
    for s, (n, q) in enumerate(zip(ctx, qlen)):
        p = torch.arange(n - q, n, device=DEV)
        lo = torch.tensor(begin[at:at + q], device=DEV) if begin else torch.zeros_like(p)
        hi = torch.tensor(end[at:at + q], device=DEV) if end else p + 1
        if W:
            lo = torch.maximum(lo, p + 1 - W)
        blocks = st["block_tables"][s, :_blocks_of(n, B)].long()
        for h in range(Hkv):
            kv = []
            for pool, scale in ((st["key_cache"], st.get("k_scale")), (st["value_cache"], st.get("v_scale"))):
                x = pool[blocks, h].reshape(-1, D)[:n]
                kv.append(x.view(torch.float8_e4m3fn).double() * scale if c["type"] == "e4m3" else x.double())
            for i0 in range(0, q, 2048):
                i1 = min(q, i0 + 2048)
                k0, k1 = int(lo[i0:i1].min().clamp(min=0)), int(hi[i0:i1].max().clamp(max=n))
                if k1 <= k0:
                    continue
                j = torch.arange(k0, k1, device=DEV)
                see = (j >= lo[i0:i1, None]) & (j < hi[i0:i1, None])
                for g in range(G):
                    x = st["query"][at + i0:at + i1, h * G + g].double() @ kv[0][k0:k1].T * st["scale"]
                    if c["softcap"]:
                        x = c["softcap"] * torch.tanh(x / c["softcap"])
                    if c["alibi"]:
                        x = x - st["slopes"][h * G + g].double() * (p[i0:i1, None] - j).abs()
                    w = torch.softmax(x.masked_fill(~see, float("-inf")), -1)
                    w = torch.where(see.any(-1, keepdim=True), w, 0.0)
                    out[at + i0:at + i1, h * G + g] = w @ kv[1][k0:k1]
        at += q
    return out
