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


@pytest.mark.parametrize("scored", [False, True])
def test_a_grid_of_empty_places_beside_another_call(scored):
    """The largest grid that a call accepts, nearly all of it empty, on the third of the SMs that another call leaves for
    more than a second."""
    b, sets = batch(False, 2), [{0, i} for i in range(Q)]
    seqs = 13  # 104 CTAs of the long rows
    mask = i32([[sum(1 << u for u in x)] for x in sets] * seqs)
    q = b["q"].repeat(seqs, 1, 1).to(DEV)
    k, v = b["k"].to(DEV), b["v"].to(DEV)
    tables = torch.stack([b["tables"][0]] * seqs).to(torch.int32).to(DEV)
    busy, out = torch.full_like(q, 7.0), torch.full((48, 8, D), 7.0, dtype=q.dtype, device=DEV)
    n, ql, blocks = 65535, 48, 256  # sequences (the last one has all tokens), their tokens, partitions of a block each
    few = torch.zeros((n, blocks), dtype=torch.int32, device=DEV)
    few[-1] = torch.arange(blocks, device=DEV) % 50
    ctx, starts = i32([0] * n), i32([0] * (n + 1))
    ctx[-1], starts[-1] = blocks * B, ql
    few_q = torch.randn((ql, 8, D), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    lens = (i32([LONG] * seqs), i32([Q * s for s in range(seqs + 1)]))
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    full = i32([[-1, -1]] * ql)
    kw = dict(max_query_len=ql, max_context_len=blocks * B, partition_size=B)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    binding.paged_attention_tree(busy, q, k, v, tables, *lens, mask, D ** -0.5, max_query_len=Q, max_context_len=LONG,
                                 workspace=small, stream=streams[0])
    if scored:
        binding.paged_attention_multi_query_scored(out, few_q, k, v, few, ctx, starts, D ** -0.5, stream=streams[1],
                                                   key_end=i32([blocks * B] * ql), **kw)
    else:
        binding.paged_attention_tree(out, few_q, k, v, few, ctx, starts, full, D ** -0.5, stream=streams[1], **kw)
    torch.cuda.synchronize()
    assert binding.device_errors() == 0
    want = torch.empty_like(out)
    args = (want, few_q, k, v, few[-1:], ctx[-1:], i32([0, ql]))
    if scored:
        binding.paged_attention_multi_query_scored(*args, D ** -0.5, key_end=i32([blocks * B] * ql), **kw)
    else:
        binding.paged_attention_tree(*args, full, D ** -0.5, **kw)
    assert torch.isfinite(out).all() and torch.equal(out, want)
