"""Inputs and the 64-bit definition for the tests of scored paged attention.

``build`` makes a batch over a shuffled pool whose unused slots hold NaN. ``reference`` computes the
definition in float64, token by token over the visible keys only, and with it the largest error that the
formats allow:

  tol = u_out |o| + sum_j p_j (|V_j| + |o|) (u_p + d_j) + floor

u_out and u_p are half steps of the output's type and of the weights' 16-bit type (finfo.eps / 2). The
normaliser's own rounding is the |o| in the sum. d_j bounds a weight's relative error from its score: the
product's sum of D terms in fp32 (D + 8 roundings of 2^-23, tensor cores truncate), the tanh (relative 1e-6),
and the fp32 exponent and reference (2^-22 of each plus one unit). The floor is the smallest steps of the
types: weights below f16's normal range (2^-25 each against a largest weight of at least 1) and the output's.
"""
import math

import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def build(seed, ctx, qlens, H, Hkv, D, B, dtype="bf16", fp8=False, spread=2.0):
    """qlens None: decode. Everything on the CPU; the pool as float64 values beside the stored one."""
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    S = len(ctx)
    q = [1] * S if qlens is None else list(qlens)
    nblk = [-(-n // B) for n in ctx]
    NB = sum(nblk) + 3
    perm = torch.randperm(NB, generator=g).tolist()
    width = max([1] + nblk)
    tables = torch.full((S, width), -1, dtype=torch.int32)
    for s, n in enumerate(nblk):
        for j in range(n):
            tables[s, j] = perm.pop()
    b = dict(ctx=list(ctx), qlens=q, decode=qlens is None, H=H, Hkv=Hkv, D=D, B=B, dtype=dt, fp8=fp8,
             scale=D ** -0.5, tables=tables, k_scale=1.0, v_scale=1.0)
    pools = []
    for name, scale in (("k", 0.02), ("v", 0.015)):
        x = torch.randn((NB, Hkv, B, D), generator=g)
        if fp8:
            code = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            nan = 0x7F
            b[name + "_scale"] = scale
        else:
            code, nan = x.to(dt), float("nan")
        used = torch.zeros(NB, B, dtype=torch.bool)
        for s, n in enumerate(ctx):
            for j in range(nblk[s]):
                used[tables[s, j], :min(B, n - j * B)] = True
        code[~used[:, None, :].expand(NB, Hkv, B)] = nan
        pools.append(code)
    b["kc"], b["vc"] = pools
    b["q"] = (torch.randn((sum(q), H, D), generator=g) * spread).to(dt)
    starts = [0]
    for k in q:
        starts.append(starts[-1] + k)
    b["starts"] = starts
    return b


def values(b, pool, scale):
    return pool.view(torch.float8_e4m3fn).double() * scale if b["fp8"] else pool.double()


def reference(b, softcap=0.0, slopes=None, window=0, key_begin=None, key_end=None):
    """(out, tol) in float64. Keys in blocks outside the pool do not take part."""
    H, Hkv, D, B = b["H"], b["Hkv"], b["D"], b["B"]
    G = H // Hkv
    NB = b["kc"].shape[0]
    kc, vc = values(b, b["kc"], b["k_scale"]), values(b, b["vc"], b["v_scale"])
    u_out = torch.finfo(b["dtype"]).eps / 2
    p16 = torch.float16 if b["fp8"] else b["dtype"]
    u_p = torch.finfo(p16).eps / 2
    out = torch.zeros((b["q"].shape[0], H, D), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for s, (n, ql) in enumerate(zip(b["ctx"], b["qlens"])):
        for i in range(ql):
            t, p = b["starts"][s] + i, n - ql + i
            lo = max(0, p - window + 1 if window else 0, key_begin[t] if key_begin is not None else 0)
            hi = min(n, key_end[t]) if key_end is not None else p + 1
            js = [j for j in range(lo, hi) if 0 <= int(b["tables"][s, j // B]) < NB]
            if not js:
                continue
            j = torch.tensor(js)
            blk, off = b["tables"][s][j // B].long(), j % B
            k, v = kc[blk, :, off], vc[blk, :, off]  # [n][Hkv][D]
            k, v = (x.repeat_interleave(G, 1) for x in (k, v))  # [n][H][D]
            qt = b["q"][t].double()
            x = torch.einsum("hd,nhd->hn", qt, k) * b["scale"]
            sabs = torch.einsum("hd,nhd->hn", qt.abs(), k.abs()) * b["scale"]
            d = (D + 8) * 2.0 ** -23 * sabs
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                d = d + 1e-6 * x.abs()
            if slopes is not None:
                x = x - slopes.double()[:, None] * (p - j).abs()
            m = x.amax(1, keepdim=True)
            d = d + 2.0 ** -22 * (x.abs() + m.abs() + 1)
            w = torch.softmax(x, 1)
            o = torch.einsum("hn,nhd->hd", w, v)
            out[t] = o
            e = w * (u_p + d + len(js) * 2.0 ** -24)
            tol[t] = (u_out * o.abs() + torch.einsum("hn,nhd->hd", e, v.abs()) + e.sum(1, keepdim=True) * o.abs()
                      + (len(js) * 2.0 ** -25 * v.abs().amax(0) if p16 is torch.float16 else 0)
                      + torch.finfo(b["dtype"]).smallest_normal * u_out * 2)
    return out, tol


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32)


def documents(b, seed):
    """Per query token the first position of its document: each sequence a row of documents of random lengths."""
    g = torch.Generator().manual_seed(seed)
    begin = []
    for n, ql in zip(b["ctx"], b["qlens"]):
        at, start, left = [], 0, 0
        for j in range(n):
            if left == 0:
                start, left = j, 1 + int(torch.randint(0, max(1, n // 3), (1,), generator=g))
            left -= 1
            at.append(start)
        begin += at[n - ql:] if ql else []
        if b["decode"] and n == 0:
            begin.append(0)
    return begin


def prefixes(b, seed):
    """Per query token the end of its visible keys under a prefix mask."""
    g = torch.Generator().manual_seed(seed)
    end = []
    for n, ql in zip(b["ctx"], b["qlens"]):
        prefix = int(torch.randint(0, n + 1, (1,), generator=g))
        end += [max(n - ql + i + 1, prefix) for i in range(ql)]
    return end


def worst(got, ref, tol):
    """The largest error in units of the tolerance."""
    got = got.double().cpu()
    assert torch.isfinite(got).all(), "non-finite output"
    return float(((got - ref).abs() / tol.clamp(min=1e-30)).max()) if got.numel() else 0.0


def ceil_div(a, b):
    return math.ceil(a / b)
