"""Drafted trees and the 64-bit definition for the tests of tree attention (the batches and the tolerance are those of
tests/scored_reference.py)."""
import random

import torch

import scored_reference as R


def parents(seed, q, roots=1, shape="tree"):
    """Each node's parent, -1 for a root."""
    r = random.Random(seed)
    if shape == "chain":
        return [i - 1 for i in range(q)]
    if shape == "star":
        return [-1 if i == 0 else 0 for i in range(q)]
    return [-1 if i < roots else max(r.randrange(i), r.randrange(i)) for i in range(q)]


def ancestors(par):
    """Each node's visible nodes: itself and its ancestors."""
    got = []
    for i, p in enumerate(par):
        got.append((got[p] if p >= 0 else set()) | {i})
    return got


def words_of(sets, W):
    """Mask rows as int32 words."""
    rows = []
    for s in sets:
        bits = sum(1 << u for u in s)
        row = [(bits >> (32 * w)) & 0xFFFFFFFF for w in range(W)]
        rows.append([x - (1 << 32) if x >= 1 << 31 else x for x in row])
    return torch.tensor(rows, dtype=torch.int32).reshape(len(rows), W)


def build(seed, committed, qlens, H, Hkv, D, B, dtype="bf16", fp8=False, shape="tree", roots=1, spread=2.0, W=None):
    """A batch of R.build whose last qlens[s] tokens are a tree; adds the parents, the visible sets and the mask."""
    b = R.build(seed, [n + q for n, q in zip(committed, qlens)], qlens, H, Hkv, D, B, dtype, fp8, spread)
    b["committed"] = list(committed)
    b["parents"] = [parents(seed * 1000 + s, q, roots, shape) for s, q in enumerate(qlens)]
    return set_mask(b, [v for p in b["parents"] for v in ancestors(p)], W)


def set_mask(b, sets, W=None):
    b["sets"] = sets
    b["W"] = W or max(1, R.ceil_div(max(b["qlens"] + [1]), 32))
    b["mask"] = words_of(sets, b["W"])
    return b


def reference(b, softcap=0.0, key_begin=None):
    """(out, tol) in float64, token by token over the visible keys; keys in blocks outside the pool do not take part."""
    H, Hkv, D, B = b["H"], b["Hkv"], b["D"], b["B"]
    G, NB = H // Hkv, b["kc"].shape[0]
    kc, vc = R.values(b, b["kc"], b["k_scale"]), R.values(b, b["vc"], b["v_scale"])
    u_out = torch.finfo(b["dtype"]).eps / 2
    p16 = torch.float16 if b["fp8"] else b["dtype"]
    u_p = torch.finfo(p16).eps / 2
    out = torch.zeros((b["q"].shape[0], H, D), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for s, (c, ql) in enumerate(zip(b["committed"], b["qlens"])):
        for i in range(ql):
            t = b["starts"][s] + i
            lo = key_begin[t] if key_begin is not None else 0
            js = [j for j in list(range(c)) + sorted(c + u for u in b["sets"][t] if u < ql) if j >= lo]
            js = [j for j in js if 0 <= int(b["tables"][s, j // B]) < NB]
            if not js:
                continue
            j = torch.tensor(js)
            blk, off = b["tables"][s][j // B].long(), j % B
            k, v = (x[blk, :, off].repeat_interleave(G, 1) for x in (kc, vc))  # [n][H][D]
            qt = b["q"][t].double()
            x = torch.einsum("hd,nhd->hn", qt, k) * b["scale"]
            d = (D + 8) * 2.0 ** -23 * torch.einsum("hd,nhd->hn", qt.abs(), k.abs()) * abs(b["scale"])
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                d = d + 1e-6 * x.abs()
            d = d + 2.0 ** -22 * (x.abs() + x.amax(1, keepdim=True).abs() + 1)
            w = torch.softmax(x, 1)
            o = torch.einsum("hn,nhd->hd", w, v)
            e = w * (u_p + d + len(js) * 2.0 ** -24)
            out[t] = o
            tol[t] = (u_out * o.abs() + torch.einsum("hn,nhd->hd", e, v.abs()) + e.sum(1, keepdim=True) * o.abs()
                      + (len(js) * 2.0 ** -25 * v.abs().amax(0) if p16 is torch.float16 else 0)
                      + torch.finfo(b["dtype"]).smallest_normal * u_out * 2)
    return out, tol
