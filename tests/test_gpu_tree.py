"""Attention of drafted trees on the GPU against the definition in 64 bits, within the error that the formats allow
(tests/tree_reference.py)."""
import random

import pytest
import torch

import scored_reference as R
import tree_reference as TR
from paged_kv_cache_91_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HIDE = (1 << 31) - 1


@pytest.fixture(autouse=True)
def clean_error_word(cuda_lib):
    binding.device_errors(clear=True)
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def call(b, softcap=0.0, key_begin=None, out=None, max_ctx=None, **kw):
    out = torch.full_like(b["q"], float("nan"), device=DEV) if out is None else out
    args = [out, b["q"].to(DEV), b["kc"].to(DEV), b["vc"].to(DEV), b["tables"].to(DEV), i32(b["ctx"]), i32(b["starts"]),
            b["mask"].to(DEV), b["scale"]]
    kw = dict(kw, softcap=softcap, key_begin=None if key_begin is None else i32(key_begin),
              max_context_len=max(b["ctx"]) if max_ctx is None else max_ctx)
    kw.setdefault("max_query_len", max(b["qlens"]))
    if b["fp8"]:
        binding.paged_attention_tree_fp8(*args, b["k_scale"], b["v_scale"], **kw)
    else:
        binding.paged_attention_tree(*args, **kw)
    torch.cuda.synchronize()
    return out


def check(b, errors=0, part=0, **rules):
    ref, tol = TR.reference(b, **rules)
    out = call(b, partition_size=part, **rules)
    assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == errors


SHAPES = [  # H, Hkv, D, B, dtype, fp8
    (4, 4, 64, 16, "f16", False), (8, 2, 128, 16, "bf16", False), (6, 2, 64, 8, "bf16", False),
    (8, 8, 128, 32, "f16", False), (16, 1, 128, 8, "f16", False), (20, 4, 128, 16, "bf16", False),
    (8, 1, 128, 16, "bf16", True), (4, 4, 128, 8, "f16", True), (24, 2, 128, 32, "bf16", True),
]
BATCHES = [  # committed tokens, drafted tokens
    ([0, 1, 15, 60], [1, 3, 2, 1]),              # single tokens, and a tree with nothing before it
    ([0, 5, 31, 100, 250], [9, 0, 12, 7, 16]),   # no token at all among them
    ([13, 129, 300], [33, 64, 40]),              # trees that pass a word of the mask and a tile of keys
]


@pytest.mark.parametrize("rule", ["none", "cap", "begin", "all"])
@pytest.mark.parametrize("committed,qlens", BATCHES)
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", SHAPES)
def test_tree(H, Hkv, D, B, dtype, fp8, committed, qlens, rule):
    b = TR.build(31, committed, qlens, H, Hkv, D, B, dtype, fp8, roots=2)
    rules = {}
    if rule in ("cap", "all"):
        rules["softcap"] = 3.0  # the scores' spread is about 2: both sides of the tanh's bend
    if rule in ("begin", "all"):  # a window of 40 positions
        rules["key_begin"] = [max(0, c + len(v) - 40) for c, q, at in zip(committed, qlens, b["starts"])
                              for v in b["sets"][at:at + q]]
    check(b, **rules)


@pytest.mark.parametrize("q", [1, 2, 7, 31, 32, 33, 95, 130, 257])
@pytest.mark.parametrize("shape", ["chain", "star", "tree"])
@pytest.mark.parametrize("fp8", [False, True])
def test_shapes_of_trees(q, shape, fp8):
    """From one token to several row tiles, and mask words that no token needs."""
    b = TR.build(32, [77, 3], [q, max(1, q // 2)], 4, 2, 128, 16, fp8=fp8, shape=shape, W=R.ceil_div(q, 32) + q % 2)
    check(b)


@pytest.mark.parametrize("part", [64, 128])
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [SHAPES[0], SHAPES[1], SHAPES[5], SHAPES[6]])
def test_split(H, Hkv, D, B, dtype, fp8, part):
    """Contexts of several partitions; drafted tokens on both sides of a border, and partitions of hidden ones alone."""
    b = TR.build(33, [60, 700, 127, 3], [8, 150, 3, 140], H, Hkv, D, B, dtype, fp8, shape="star")
    check(b, part=part)
    ref, tol = TR.reference(b, softcap=4.0)
    out = call(b, partition_size=part, max_ctx=b["tables"].shape[1] * B, softcap=4.0)
    assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[3, 2], [70, 90]])
def test_any_mask(qlens, fp8):
    """Masks of no tree: rows that see nothing drafted, not themselves, everything, and bits past the tree."""
    b = TR.build(34, [0, 90], qlens, 4, 2, 128, 16, fp8=fp8)
    sets = [set() if i % 3 == 0 else set(range(q)) | {q, 95} if i % 3 == 1 else {q - 1}
            for q in qlens for i in range(q)]
    check(TR.set_mask(b, sets, W=3))


@pytest.mark.parametrize("q", [2, 60])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_see_nothing(q, fp8):
    """A sequence that waits (everything hidden; its drafted tokens have no blocks), rows hidden among others, and
    a first key among the drafted ones."""
    b = TR.build(35, [60, 16, 200], [q, q, q], 8, 2, 128, 16, fp8=fp8)
    b["tables"][1, 1:] = -1
    begin = [-(1 << 31) if i % 2 else 61 for i in range(q)] + [HIDE] * q + [HIDE if i % 3 == 0 else 199 for i in range(q)]
    check(b, key_begin=begin)
    check(b, key_begin=begin, softcap=2.0, part=64)
    check(b, key_begin=[HIDE] * (3 * q))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens,part", [([5, 4], 0), ([60, 90], 0), ([60, 90], 64)])
def test_a_hidden_key_may_hold_anything(qlens, part, fp8):
    """NaN and infinities in drafted keys that some rows see do not reach the rows that do not see them."""
    b = TR.build(36, [40, 150], qlens, 4, 2, 128, 16, "bf16", fp8, shape="star")
    bad = [(0, 40 + 2, float("nan")), (1, 150 + 3, float("inf"))]
    for s, at, x in bad:
        for pool in (b["kc"], b["vc"]) if x != x else (b["vc"],):
            pool[b["tables"][s, at // 16], :, at % 16] = 0x7F if fp8 else x
    for rules in (dict(), dict(softcap=5.0)):
        ref, tol = TR.reference(b, **rules)
        out = call(b, partition_size=part, **rules).double().cpu()
        seen = [at + bad[s][1] - b["committed"][s] for s, at in enumerate(b["starts"][:2])]
        blind = [t for t in range(sum(qlens)) if t not in seen]
        assert R.worst(out[blind], ref[blind], tol[blind]) <= 1.0
        assert not torch.isfinite(out[seen]).all(dim=-1).any()


def test_a_chain_is_causal_attention():
    """On the chain's mask the call's definition is paged_attention_multi_query_scored's."""
    for qlens in ([3, 2, 4], [50, 64, 7]):
        b = TR.build(37, [100, 0, 333], qlens, 8, 2, 128, 16, shape="chain")
        want = torch.empty_like(b["q"], device=DEV)
        binding.paged_attention_multi_query_scored(
            want, b["q"].to(DEV), b["kc"].to(DEV), b["vc"].to(DEV), b["tables"].to(DEV), i32(b["ctx"]),
            i32(b["starts"]), b["scale"], softcap=5.0, max_query_len=max(qlens), max_context_len=max(b["ctx"]))
        ref, tol = TR.reference(b, softcap=5.0)
        assert R.worst(want, ref, tol) <= 1.0
        assert R.worst(call(b, softcap=5.0), ref, tol) <= 1.0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q", [4, 40])
def test_bad_block_ids_are_skipped_and_reported(q, fp8):
    b = TR.build(38, [100, 50], [q, q], 4, 2, 128, 16, fp8=fp8)
    b["tables"][0, 2] = -7
    b["tables"][1, (50 + q - 1) // 16] = b["kc"].shape[0]
    check(b, errors=1)


@pytest.mark.parametrize("q", [4, 40])
def test_bad_offsets_skip_their_sequence(q):
    b = TR.build(39, [100, 50, 20], [q, q, q], 4, 2, 128, 16)
    ref, tol = TR.reference(b)
    out = torch.full_like(b["q"], 7.0, device=DEV)
    b["ctx"][1] = q - 1  # fewer than its drafted tokens
    call(b, out=out, max_ctx=b["tables"].shape[1] * 16)
    keep = list(range(q)) + list(range(2 * q, 3 * q))
    assert R.worst(out[keep], ref[keep], tol[keep]) <= 1.0
    assert (out[q:2 * q] == 7.0).all()
    assert binding.device_errors() == 16


@pytest.mark.parametrize("q", [3, 50])
def test_rows_behind_the_last_sequence_are_left(q):
    """A padded batch: query, out and mask have more rows than the sequences' tokens."""
    b = TR.build(40, [90, 33], [q, q], 4, 2, 128, 16)
    ref, tol = TR.reference(b)
    b["q"] = torch.cat([b["q"], torch.full((5, 4, 128), float("nan"), dtype=b["dtype"])])
    b["mask"] = torch.cat([b["mask"], torch.full((5, b["W"]), -1, dtype=torch.int32)])
    out = torch.full_like(b["q"], 7.0, device=DEV)
    call(b, out=out)
    assert R.worst(out[:2 * q], ref, tol) <= 1.0 and (out[2 * q:] == 7.0).all()


@pytest.mark.parametrize("q,part", [(3, 0), (3, 64), (40, 0), (40, 64)])
def test_captured_and_replayed(q, part):
    """Replays follow what their buffers hold, and two graphs with one workspace run one after the other."""
    first, second = (TR.build(s, [300, 120], [q, q], 8, 2, 128, 16) for s in (41, 42))
    dev = {k: first[k].to(DEV) for k in ("q", "kc", "vc", "tables", "mask")}
    ctx, starts, outs = i32(first["ctx"]), i32(first["starts"]), [torch.empty_like(dev["q"]) for _ in range(2)]
    need = binding.paged_attention_tree_workspace_size(2 * q, 8, 2, 128, 16, q, max(first["ctx"]), part)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)

    def step(out):
        binding.paged_attention_tree(out, dev["q"], dev["kc"], dev["vc"], dev["tables"], ctx, starts, dev["mask"],
                                     first["scale"], max_query_len=q, max_context_len=max(first["ctx"]),
                                     partition_size=part, workspace=ws)

    step(outs[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in outs]
    for g, out in zip(graphs, outs):
        with torch.cuda.graph(g):
            step(out)
    for b in (first, second, first):
        for k, t in dev.items():
            t.copy_(b[k])
        for out in outs:
            out.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ref, tol = TR.reference(b)
        for out in outs:
            assert R.worst(out, ref, tol) <= 1.0


def test_on_another_stream_and_repeated():
    """The call's own workspace and its work are on the given stream; the same call gives the same bits."""
    b = TR.build(43, [900, 700, 5], [30, 64, 12], 8, 2, 128, 16)
    want = call(b, partition_size=128)
    side = torch.cuda.Stream()
    for _ in range(3):
        out = torch.full_like(want, float("nan"))
        torch.cuda.synchronize()
        call(b, out=out, partition_size=128, stream=side)
        assert torch.equal(out, want)
    assert binding.device_errors() == 0


@pytest.mark.parametrize("q", [2, 40])
def test_a_long_cache(q):
    """A pool of more than 2^31 bytes, whose blocks lie at its end."""
    H, Hkv, D, B = 8, 8, 128, 32
    b = TR.build(44, [500], [q], H, Hkv, D, B)
    NB = (1 << 31) // (Hkv * B * D * 2) + 200
    used = b["kc"].shape[0]
    pools = [torch.zeros((NB, Hkv, B, D), dtype=b["dtype"], device=DEV) for _ in range(2)]
    for pool, small in zip(pools, (b["kc"], b["vc"])):
        pool[NB - used:] = small.to(DEV)
    ref, tol = TR.reference(b)
    out = torch.empty_like(b["q"], device=DEV)
    tables = torch.where(b["tables"] >= 0, b["tables"] + (NB - used), b["tables"])
    binding.paged_attention_tree(out, b["q"].to(DEV), *pools, tables.to(DEV), i32(b["ctx"]), i32(b["starts"]),
                                 b["mask"].to(DEV), b["scale"], max_query_len=q)
    torch.cuda.synchronize()
    assert R.worst(out, ref, tol) <= 1.0


@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [(16, 8, 128, 16, "bf16", False), (16, 8, 64, 8, "f16", False),
                                                 (16, 8, 128, 32, "bf16", True), (24, 8, 128, 16, "f16", True)])
@pytest.mark.parametrize("part", [0, 96])
def test_more_work_than_ctas(H, Hkv, D, B, dtype, fp8, part):
    """CTAs that take several items each, sequences of every length in no order: long ones, without drafted tokens, that
    wait, with nothing committed, with bad offsets."""
    r = random.Random(45)
    committed = [r.choice([0, 3, 40, 130, 400, r.randint(0, 300)]) for _ in range(46)]
    qlens = [r.choice([0, 1, 5, 6, 9]) for _ in committed]
    qlens[3], qlens[20] = 9, 70  # (several row tiles)
    b = TR.build(45, committed, qlens, H, Hkv, D, B, dtype, fp8)
    begin = [0] * sum(qlens)
    for s in (5, 6, 30, 45):
        for t in range(b["starts"][s], b["starts"][s + 1]):
            begin[t] = HIDE
        b["tables"][s] = -1
    for s in (7, 8):  # windows
        for t in range(b["starts"][s], b["starts"][s + 1]):
            begin[t] = max(0, committed[s] - 20)
    if part:
        part = part // B * B
    ref, tol = TR.reference(b, key_begin=begin)
    rows = list(range(sum(qlens)))
    out = torch.full_like(b["q"], 7.0, device=DEV)
    call(b, key_begin=begin, out=out, partition_size=part)
    assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == 0
    bad = next(s for s in range(10, 46) if qlens[s] > 1)
    b["ctx"][bad] = 1
    gone = rows[b["starts"][bad]:b["starts"][bad + 1]]
    keep = [t for t in rows if t not in gone]
    out.fill_(7.0)
    call(b, key_begin=begin, out=out, partition_size=part, max_ctx=b["tables"].shape[1] * B)
    assert R.worst(out[keep], ref[keep], tol[keep]) <= 1.0 and (out[gone] == 7.0).all()
    assert binding.device_errors() == 16


def test_more_sequences_than_are_sorted():
    r = random.Random(46)
    committed = [r.randint(0, 60) for _ in range(150)]
    b = TR.build(46, committed, [r.randint(1, 4) for _ in committed], 12, 4, 128, 16)
    check(b)
    check(b, part=32)


@pytest.mark.parametrize("q", [2, 20])
@pytest.mark.parametrize("power", [-50, 50])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 3.0])
def test_queries_of_any_size(q, power, fp8, softcap):
    """Queries far from 1 with a scale that brings the scores back, and a row of zeros."""
    b = TR.build(47, [150, 9], [q, q], 8, 2, 128, 16, fp8=fp8)
    b["q"] = b["q"] * 2.0 ** power
    b["q"][1, 3] = 0.0
    b["scale"] = 128 ** -0.5 * 2.0 ** -power
    check(b, softcap=softcap)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own."""
    bs = [TR.build(s, [700, 300, 40], [24, 30, 12], 8, 2, 128, 16) for s in (48, 49)]
    dev = [{k: b[k].to(DEV) for k in ("q", "kc", "vc", "tables", "mask")} for b in bs]
    ctx, starts = [i32(b["ctx"]) for b in bs], [i32(b["starts"]) for b in bs]
    outs, streams = [torch.empty_like(d["q"]) for d in dev], [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, b in enumerate(bs):
            d = dev[i]
            binding.paged_attention_tree(outs[i], d["q"], d["kc"], d["vc"], d["tables"], ctx[i], starts[i], d["mask"],
                                         b["scale"], max_query_len=30, max_context_len=max(b["ctx"]),
                                         partition_size=128, stream=streams[i])
    torch.cuda.synchronize()
    for b, out in zip(bs, outs):
        ref, tol = TR.reference(b)
        assert R.worst(out, ref, tol) <= 1.0


@pytest.mark.parametrize("H,Hkv,D,B,fp8", [(160, 1, 128, 16, False), (144, 1, 64, 8, False), (300, 2, 128, 32, True)])
def test_many_heads_a_kv_head(H, Hkv, D, B, fp8):
    """A token's heads pass a row tile."""
    b = TR.build(50, [70, 5], [1, 3], H, Hkv, D, B, fp8=fp8)
    check(b)
    check(b, part=64, softcap=3.0)


@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_loose_bounds(fp8, part):
    """Bounds on query tokens and contexts far above what there is: row tiles and partitions without work."""
    b = TR.build(51, [0, 300, 21], [2, 9, 0], 8, 2, 128, 16, fp8=fp8, W=13)
    b["tables"] = torch.cat([b["tables"], torch.full((3, 200), -1, dtype=torch.int32)], 1)
    ref, tol = TR.reference(b)
    out = call(b, partition_size=part, max_query_len=400, max_ctx=b["tables"].shape[1] * 16)
    assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == 0


@pytest.mark.parametrize("q", [2, 40])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [-0.09, 0.0])
def test_scales_that_are_not_positive(q, fp8, scale):
    b = TR.build(52, [150, 9], [q, q], 8, 2, 128, 16, fp8=fp8)
    b["scale"] = scale
    check(b)
    check(b, softcap=3.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_workspace_of_any_size(fp8):
    """The partitions are as many as the workspace holds."""
    b = TR.build(53, [2500], [20], 8, 2, 128, 16, fp8=fp8)
    ref, tol = TR.reference(b)
    need = binding.paged_attention_tree_workspace_size(20, 8, 2, 128, 16, 20, 2520)
    assert need > 0
    for size in (need, need // 2, need // 3, 16):
        out = call(b, workspace=torch.empty(size, dtype=torch.uint8, device=DEV))
        assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == 0


def test_a_large_tree():
    """More nodes than a mask of paged_kv_tree_layout holds."""
    b = TR.build(54, [17], [1100], 2, 1, 64, 16, "f16")
    check(b)
