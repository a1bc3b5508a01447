"""Rows of long contexts that are computed again because a key that they do not see holds a NaN: a warp's rows take more
than a second, longer than any wait in the kernels may last without a sign of work.

A context of 130,000 tokens is a table that names 60 blocks over and over, so that the definition is a sum over each
block's keys times how often it is named. The tolerance is that of tests/scored_reference.py."""
import pytest
import torch

from paged_kv_cache_91_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, HKV, D, B, NB, Q = 64, 8, 128, 32, 64, 16
LONG, SHORT = 130_048 + Q, 64 + Q  # Q new tokens behind whole blocks
SEQS = 20  # 19 long ones fill 152 CTAs with an item each; the short one's items come after them


@pytest.fixture(autouse=True)
def clean_error_word(cuda_lib):
    binding.device_errors(clear=True)
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def batch(fp8, bad):
    """bad: the new token of the long sequences whose value is NaN."""
    g = torch.Generator().manual_seed(71)
    k, v = (torch.randn((NB, HKV, B, D), generator=g) for _ in range(2))
    b = dict(fp8=fp8, scales=(0.02, 0.015) if fp8 else (), q=(2 * torch.randn((Q, H, D), generator=g)).bfloat16())
    long = torch.cat([torch.randint(0, 60, ((LONG - Q) // B,), generator=g), torch.tensor([60])])
    short = torch.full_like(long, -1)
    short[:3] = torch.tensor([3, 1, 61])
    b["tables"] = [long, short]
    for name, x, scale in (("k", k, 0.02), ("v", v, 0.015)):
        if fp8:
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            b[name] = x.view(torch.uint8)
        else:
            b[name] = x.bfloat16()
    b["v"][60, :, bad] = 0x7F if fp8 else float("nan")
    b["kd"], b["vd"] = (x.view(torch.float8_e4m3fn).double() * s if fp8 else x.double()
                        for x, s in ((b["k"], 0.02), (b["v"], 0.015)))
    return b


def definition(b, table, n, sets):
    """(out, tol) [Q][H][D] of the new tokens, token i seeing the committed ones and the new ones of sets[i]."""
    u_out, u_p = (torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16 if b["fp8"] else torch.bfloat16))
    scale, out, tol = D ** -0.5, [], []
    for i in range(Q):
        times = torch.bincount(table[:(n - Q) // B], minlength=NB).double()[:, None].repeat(1, B)
        for u in sets[i]:
            times[table[(n - Q) // B], u] += 1
        blk, off = torch.nonzero(times, as_tuple=True)
        times = times[blk, off]
        k, v = (x[blk, :, off].repeat_interleave(H // HKV, 1) for x in (b["kd"], b["vd"]))
        q = b["q"][i].double()
        x = torch.einsum("hd,nhd->hn", q, k) * scale
        d = (D + 8) * 2.0 ** -23 * torch.einsum("hd,nhd->hn", q.abs(), k.abs()) * scale
        d = d + 2.0 ** -22 * (x.abs() + x.amax(1, keepdim=True).abs() + 1)
        w = torch.softmax(x + times.log(), 1)
        o = torch.einsum("hn,nhd->hd", w, v)
        e = w * (u_p + d + n * 2.0 ** -24)
        out.append(o)
        tol.append(u_out * o.abs() + torch.einsum("hn,nhd->hd", e, v.abs()) + e.sum(1, keepdim=True) * o.abs()
                   + (n * 2.0 ** -25 * v.abs().amax(0) if b["fp8"] else 0))
    return torch.stack(out), torch.stack(tol)


def check(b, sets, bad, call):
    tables = torch.stack([b["tables"][0]] * (SEQS - 1) + [b["tables"][1]]).to(torch.int32).to(DEV)
    q = b["q"].repeat(SEQS, 1, 1).to(DEV)
    out = torch.full_like(q, 7.0)
    call(out, q, b["k"].to(DEV), b["v"].to(DEV), tables, i32([LONG] * (SEQS - 1) + [SHORT]),
         i32([Q * s for s in range(SEQS + 1)]))
    torch.cuda.synchronize()
    assert binding.device_errors() == 0
    got = out.double().cpu().reshape(SEQS, Q, H, D)
    for s, n, table in ((0, LONG, 0), (SEQS - 2, LONG, 0), (SEQS - 1, SHORT, 1)):
        ref, tol = definition(b, b["tables"][table], n, sets)
        seen = [i for i in range(Q) if table == 0 and bad in sets[i]]
        blind = [i for i in range(Q) if i not in seen]
        assert float(((got[s] - ref).abs() / tol)[blind].max()) <= 1.0
        assert not torch.isfinite(got[s, seen]).all(dim=-1).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_tree(fp8):
    bad = 2
    b = batch(fp8, bad)
    sets = [{0, i} for i in range(Q)]
    mask = i32([[sum(1 << u for u in x)] for x in sets] * SEQS)

    def call(out, q, k, v, tables, ctx, starts):
        fn = binding.paged_attention_tree_fp8 if fp8 else binding.paged_attention_tree
        fn(out, q, k, v, tables, ctx, starts, mask, D ** -0.5, *b["scales"], max_query_len=Q, max_context_len=LONG,
           workspace=torch.empty(16, dtype=torch.uint8, device=DEV))  # (one partition a sequence)

    check(b, sets, bad, call)


def test_scored():
    bad = Q - 1
    b = batch(False, bad)

    def call(out, q, k, v, tables, ctx, starts):
        binding.paged_attention_multi_query_scored(
            out, q, k, v, tables, ctx, starts, D ** -0.5, max_query_len=Q, max_context_len=LONG,
            workspace=torch.empty(16, dtype=torch.uint8, device=DEV))

    check(b, [set(range(i + 1)) for i in range(Q)], bad, call)
