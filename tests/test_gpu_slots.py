"""Block tables and slot maps built on the GPU (paged_kv_reserve_slots, paged_kv_release_blocks) against the rule
in plain Python; whole numbers, compared exactly. And a serving loop of reserve, cache write, scored attention
and release."""
import random

import pytest
import torch

import scored_reference as R
from paged_kv_cache_91_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def clean_error_word(cuda_lib):
    binding.device_errors(clear=True)
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def reserve_rule(tables, ctx, new, free, nfree, B, max_tokens):
    tables, taken = [list(r) for r in tables], 0
    cum, granted, ctx_out, slots, starts = 0, [], [], [], [0]
    for s, (n, k) in enumerate(zip(ctx, new)):
        have, need = -(-n // B), -(-(n + k) // B) - -(-n // B)
        cum += need
        ok = need == 0 or cum <= nfree
        if ok:
            for j in range(need):
                tables[s][have + j] = free[nfree - 1 - taken]
                taken += 1
            slots += [tables[s][p // B] * B + p % B for p in range(n, n + k)]
        else:
            slots += [-1] * k
        granted.append(int(ok))
        ctx_out.append(n + k if ok else n)
        starts.append(starts[-1] + k)
    return tables, slots + [-1] * (max_tokens - len(slots)), starts, ctx_out, [nfree - taken], granted


def make_pool(seed, ctx, room, B, spare):
    """Tables of contiguous-by-turn random blocks, and the free stack above them."""
    r = random.Random(seed)
    used = [-(-n // B) for n in ctx]
    width = max([1] + [-(-(n + k) // B) for n, k in zip(ctx, room)])
    NB = sum(used) + spare
    ids = list(range(max(NB, 1)))
    r.shuffle(ids)
    tables = [[-1] * width for _ in ctx]
    for s, n in enumerate(used):
        for j in range(n):
            tables[s][j] = ids.pop()
    return tables, ids, max(NB, 1)


def reserve(tables, ctx, new, free, nfree, B, max_tokens, NB, stream=None):
    S = len(ctx)
    t = i32(tables).reshape(S, -1) if S else torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    slots = torch.full((max_tokens,), -5, dtype=torch.int64, device=DEV)
    starts, ctx_out, granted = i32([-5] * (S + 1)), i32([-5] * S), i32([-5] * S)
    free_out = i32([-5])
    binding.paged_kv_reserve_slots(t, i32(ctx), i32(new), i32(free), i32([nfree]), slots, starts, ctx_out, free_out,
                                   granted, B, NB, stream=stream)
    torch.cuda.synchronize()
    return (t.tolist(), slots.tolist(), starts.tolist(), ctx_out.tolist(), free_out.tolist(), granted.tolist())


CASES = [  # sequences, largest context, largest new length, spare blocks, padding
    (1, 0, 1, 4, 0), (1, 40, 0, 1, 3), (3, 20, 5, 30, 2), (64, 300, 1, 40, 0), (64, 300, 1, 3, 9),
    (37, 100, 90, 120, 5), (5, 500, 3000, 900, 0), (2049, 64, 3, 700, 11), (5000, 40, 1, 200, 100),
    (600, 30, 0, 1, 4),
]


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("S,hi,new_hi,spare,pad", CASES)
def test_reserve(S, hi, new_hi, spare, pad, B):
    r = random.Random(S * 1000 + hi + new_hi + B)
    ctx = [r.randint(0, hi) for _ in range(S)]
    new = [r.choice([0, new_hi, r.randint(0, new_hi)]) for _ in range(S)]
    tables, free, NB = make_pool(r.random(), ctx, new, B, spare)
    T = sum(new) + pad
    want = reserve_rule(tables, ctx, new, free, len(free), B, T)
    got = reserve(tables, ctx, new, free, len(free), B, T, NB)
    assert got == want
    assert binding.device_errors() == 0


def test_reserve_of_an_empty_batch():
    got = reserve([], [], [], [3, 4], 2, 16, 5, 8)
    assert got == ([], [-1] * 5, [0], [], [2], [])


def test_reserve_takes_part_of_the_stack():
    """num_free says how much of free_blocks is the stack; what lies above it is not handed out."""
    tables, free, NB = make_pool(1, [0, 0], [20, 20], 16, 9)
    want = reserve_rule(tables, [0, 0], [20, 20], free, 3, 16, 40)
    assert want[5] == [1, 0]
    assert reserve(tables, [0, 0], [20, 20], free, 3, 16, 40, NB) == want


def test_reserve_reports_bad_lengths():
    B, tables, free = 16, [[0, -1], [1, -1], [2, -1], [3, -1]], [4, 5, 6, 7]
    got = reserve(tables, [16, -2, 10, 16], [1, 3, 40, 2], free, 4, B, 60, 8)
    assert got[2] == [0, 1, 4, 44, 46] and got[3] == [17, -2, 10, 18] and got[5] == [1, 0, 0, 1]
    assert got[1] == [7 * 16] + [-1] * 43 + [6 * 16, 6 * 16 + 1] + [-1] * 14
    assert binding.device_errors() == 2
    got = reserve(tables, [16, 3, 10, 16], [1, -3, 1, 2], free, 4, B, 4, 8)
    assert got[2] == [0, 1, 1, 2, 4] and got[5] == [1, 0, 1, 1]
    assert binding.device_errors() == 2


def test_reserve_reports_too_many_tokens():
    tables, free = [[0, -1], [1, -1], [2, -1]], [4, 5, 6, 7]
    got = reserve(tables, [16, 10, 5], [1, 4, 2], free, 4, 16, 4, 8)
    assert got[1] == [7 * 16, -1, -1, -1] and got[5] == [1, 0, 0] and got[2] == [0, 1, 4, 4] and got[4] == [3]
    assert binding.device_errors() == 16


def test_reserve_grants_a_sequence_without_tokens_behind_the_last_place():
    """Only a sequence with tokens past max_tokens is refused: one that asks for none needs none."""
    tables, free = [[0, -1], [1, -1], [2, -1], [3, -1]], [4, 5, 6, 7]
    got = reserve(tables, [16, 10, 5, 0], [1, 4, 0, 0], free, 4, 16, 4, 8)
    assert got[1] == [7 * 16, -1, -1, -1] and got[2] == [0, 1, 4, 4, 4]
    assert got[3] == [17, 10, 5, 0] and got[4] == [3] and got[5] == [1, 0, 1, 1]
    assert binding.device_errors() == 16


def test_reserve_reports_bad_ids():
    got = reserve([[0, -1], [9, -1], [-1, -1]], [16, 5, 3], [1, 1, 1], [1, 2, 77], 3, 16, 3, 8)
    assert got[0] == [[0, -1], [9, -1], [-1, -1]] and got[1] == [-1, -1, -1]
    assert binding.device_errors() == 1
    got = reserve([[0, -1]], [16], [1], [1, 2], 5, 16, 1, 8)  # more free blocks than the stack can hold: clamped
    assert got[1] == [2 * 16] and got[4] == [1]
    assert binding.device_errors() == 1
    got = reserve([[0, -1]], [16], [1], [1, 2], -5, 16, 1, 8)
    assert got[1] == [-1] and got[4] == [0] and got[5] == [0]
    assert binding.device_errors() == 1


def release(tables, ctx, gone, stack, nfree, B, NB):
    S = len(ctx)
    t = i32(tables).reshape(S, -1) if S else torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    free, ctx_out, free_out = i32(stack), i32([-5] * S), i32([-5])
    binding.paged_kv_release_blocks(t, i32(ctx), i32(gone), free, i32([nfree]), ctx_out, free_out, B, NB)
    torch.cuda.synchronize()
    return free.tolist(), ctx_out.tolist(), free_out.tolist()


def release_rule(tables, ctx, gone, stack, nfree, B):
    stack = list(stack)
    for s, (n, f) in enumerate(zip(ctx, gone)):
        if f:
            for j in range(-(-n // B)):
                stack[nfree] = tables[s][j]
                nfree += 1
    return stack, [0 if f else n for n, f in zip(ctx, gone)], [nfree]


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("S,hi,share", [(1, 40, 1.0), (3, 0, 1.0), (64, 300, 0.3), (700, 200, 0.5), (5000, 64, 1.0),
                                        (2, 9000, 1.0), (300, 500, 0.0)])
def test_release(S, hi, share, B):
    r = random.Random(S + hi + B)
    ctx = [r.randint(0, hi) for _ in range(S)]
    gone = [r.choice([1, -1, 7]) if r.random() < share else 0 for _ in range(S)]
    tables, free, NB = make_pool(r.random(), ctx, [0] * S, B, 5)
    stack = free + [-2] * (NB - len(free))
    assert release(tables, ctx, gone, stack, len(free), B, NB) == release_rule(tables, ctx, gone, stack, len(free), B)
    assert binding.device_errors() == 0


def test_release_of_an_empty_batch():
    assert release([], [], [], [4, 5, -2], 2, 16, 8) == ([4, 5, -2], [], [2])


def test_release_reports_bad_inputs():
    # a bad id is pushed as -1; a context past the table is clamped; blocks past the capacity are dropped
    assert release([[1, 9], [2, 3]], [32, 5], [1, 1], [-2] * 4, 0, 16, 8) == ([1, -1, 2, -2], [0, 0], [3])
    assert binding.device_errors() == 1
    assert release([[1, 4], [2, 3]], [99, -5], [1, 1], [-2] * 4, 0, 16, 8) == ([1, 4, -2, -2], [0, 0], [2])
    assert binding.device_errors() == 2
    assert release([[1, 4], [2, 3]], [32, 32], [1, 1], [-2] * 3, 0, 16, 8) == ([1, 4, 2], [0, 0], [3])
    assert binding.device_errors() == 1
    assert release([[1, 4]], [32], [1], [-2] * 3, 9, 16, 8) == ([-2] * 3, [0], [3])
    assert binding.device_errors() == 1


def test_release_then_reserve_hands_the_blocks_out_again():
    B, r = 16, random.Random(3)
    ctx = [r.randint(1, 200) for _ in range(40)]
    tables, free, NB = make_pool(4, ctx, [0] * 40, B, 0)
    gone = [int(s % 3 == 0) for s in range(40)]
    stack, ctx1, nfree = release(tables, ctx, gone, free + [-1] * (NB - len(free)), len(free), B, NB)
    new = [30 if g else 0 for g in gone]
    want = reserve_rule(tables, ctx1, new, stack, nfree[0], B, sum(new))
    assert reserve(tables, ctx1, new, stack, nfree[0], B, sum(new), NB) == want
    assert binding.device_errors() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("graphed", [False, True])
def test_serving_loop(fp8, graphed):
    """Four steps of a batch of three sequence places: prompts, decode steps, and a place that is released and
    taken by a new prompt. Each step reserves, writes the cache and attends on the GPU with no host read; the
    outputs are checked against the definition over the sequences' own keys and values."""
    S, H, Hkv, D, B, NB, T = 3, 8, 2, 128, 16, 24, 64
    scale, window, cap = D ** -0.5, 30, 4.0
    ks, vs = 0.02, 0.015
    g = torch.Generator().manual_seed(7)
    dt = torch.bfloat16
    slopes = R.slopes_of(H)
    width = 6
    nan = 0x7F if fp8 else float("nan")
    kc, vc = (torch.full((NB, Hkv, B, D), nan, dtype=torch.uint8 if fp8 else dt, device=DEV) for _ in range(2))
    dev = dict(tables=torch.full((S, width), -1, dtype=torch.int32, device=DEV), ctx=i32([0] * S), new=i32([0] * S),
               gone=i32([0] * S), free=i32(list(range(NB))), nfree=i32([NB]), nfree2=i32([0]), ctx2=i32([0] * S),
               starts=i32([0] * (S + 1)), granted=i32([0] * S), nfree3=i32([0]), ctx3=i32([0] * S),
               slots=torch.zeros(T, dtype=torch.int64, device=DEV))
    q = torch.zeros((T, H, D), dtype=dt, device=DEV)
    k, v = (torch.zeros((T, Hkv, D), dtype=dt, device=DEV) for _ in range(2))
    out = torch.zeros_like(q)
    sl = slopes.to(DEV)

    def step():
        binding.paged_kv_release_blocks(dev["tables"], dev["ctx"], dev["gone"], dev["free"], dev["nfree"],
                                        dev["ctx2"], dev["nfree2"], B, NB)
        binding.paged_kv_reserve_slots(dev["tables"], dev["ctx2"], dev["new"], dev["free"], dev["nfree2"],
                                       dev["slots"], dev["starts"], dev["ctx3"], dev["nfree3"], dev["granted"], B, NB)
        args = (out, q, kc, vc, dev["tables"], dev["ctx3"], dev["starts"], scale)
        kw = dict(softcap=cap, window=window, alibi_slopes=sl, max_query_len=40, max_context_len=width * B)
        if fp8:
            binding.paged_kv_write_fp8(k, v, kc, vc, dev["slots"], ks, vs)
            binding.paged_attention_multi_query_scored_fp8(*args, k_scale=ks, v_scale=vs, **kw)
        else:
            binding.paged_kv_write(k, v, kc, vc, dev["slots"])
            binding.paged_attention_multi_query_scored(*args, **kw)
        dev["ctx"].copy_(dev["ctx3"])
        dev["nfree"].copy_(dev["nfree3"])

    graph = None
    if graphed:
        step()  # an empty step: nothing finished, nothing new
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    hist = [dict(k=[], v=[]) for _ in range(S)]
    for new, gone in (([33, 7, 0], [0, 0, 0]), ([1, 1, 12], [0, 0, 0]), ([1, 40, 1], [0, 1, 0]),
                      ([1, 1, 1], [0, 0, 0])):
        n = sum(new)
        hq, hk, hv = (torch.randn((T, h, D), generator=g).to(dt) for h in (H, Hkv, Hkv))
        for dst, src in ((q, hq), (k, hk), (v, hv)):
            dst.copy_(src)
        dev["new"].copy_(i32(new))
        dev["gone"].copy_(i32(gone))
        out.fill_(9.0)
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        at = 0
        for s in range(S):
            if gone[s]:
                hist[s] = dict(k=[], v=[])
            hist[s]["k"] += list(hk[at:at + new[s]])
            hist[s]["v"] += list(hv[at:at + new[s]])
            at += new[s]
        ctx = [len(h["k"]) for h in hist]
        assert dev["ctx3"].tolist() == ctx and dev["granted"].tolist() == [1] * S
        b = R.build(1, ctx, new, H, Hkv, D, B, "bf16", fp8)
        if fp8:
            b.update(k_scale=ks, v_scale=vs)
        for s in range(S):
            for j in range(ctx[s]):
                for pool, name, sc in (("kc", "k", ks), ("vc", "v", vs)):
                    x = hist[s][name][j]
                    if fp8:
                        x = (x.float() / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    b[pool][b["tables"][s, j // B], :, j % B] = x
        b["q"] = hq[:n]
        ref, tol = R.reference(b, softcap=cap, window=window, slopes=slopes)
        assert R.worst(out[:n], ref, tol) <= 1.0
        assert (out[n:] == 9.0).all()
        assert binding.device_errors() == 0
    assert dev["nfree"].item() == NB - sum(-(-c // B) for c in ctx)


# New tokens and releases of each step, over pools of 3 and 6 blocks of 16 tokens.
WAITING = {
    # up to 2 query tokens a step: the tile of few rows
    "few": (3, 3, 2, [([2, 2, 0], [0, 0, 0])] * 8 + [([1, 1, 1], [0, 0, 0]), ([1, 1, 2], [0, 0, 0]),
                      ([2, 1, 1], [1, 0, 0]), ([1, 1, 2], [0, 1, 0])], 5),
    "many": (6, 4, 40, [([40, 30, 0], [0, 0, 0]), ([8, 1, 20], [0, 0, 0]), ([10, 10, 1], [0, 0, 0]),
                        ([1, 20, 40], [0, 0, 0]), ([40, 20, 1], [1, 0, 0]), ([1, 1, 16], [0, 0, 0])], 7),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("graphed", [False, True])
@pytest.mark.parametrize("rows", ["few", "many"])
def test_serving_loop_with_sequences_that_wait(fp8, graphed, rows):
    """The pool runs short: a prompt, and later a sequence at the end of its last block, wait until another one is
    released. Their query tokens have slot -1 and see no key: their rows are zeros, every other sequence's are those
    of the definition, and no error is reported; nothing is read on the host."""
    S, H, Hkv, D, B, T = 3, 8, 2, 128, 16, 96
    NB, width, longest, steps, waiting = WAITING[rows]
    scale, cap, window, ks, vs = D ** -0.5, 4.0, 30, 0.02, 0.015
    g = torch.Generator().manual_seed(9)
    dt = torch.bfloat16
    kc, vc = (torch.zeros((NB, Hkv, B, D), dtype=torch.uint8 if fp8 else dt, device=DEV) for _ in range(2))
    dev = {n: i32([0] * S) for n in ("ctx", "new", "gone", "ctx2", "granted", "ctx3", "attend")}
    dev.update(tables=torch.full((S, width), -1, dtype=torch.int32, device=DEV), free=i32(list(range(NB))),
               nfree=i32([NB]), nfree2=i32([0]), nfree3=i32([0]), starts=i32([0] * (S + 1)),
               slots=torch.zeros(T, dtype=torch.int64, device=DEV), begin=i32([0] * T))
    q = torch.zeros((T, H, D), dtype=dt, device=DEV)
    kn, vn = (torch.zeros((T, Hkv, D), dtype=dt, device=DEV) for _ in range(2))
    out = torch.zeros_like(q)

    def step():
        binding.paged_kv_release_blocks(dev["tables"], dev["ctx"], dev["gone"], dev["free"], dev["nfree"],
                                        dev["ctx2"], dev["nfree2"], B, NB)
        binding.paged_kv_reserve_slots(dev["tables"], dev["ctx2"], dev["new"], dev["free"], dev["nfree2"],
                                       dev["slots"], dev["starts"], dev["ctx3"], dev["nfree3"], dev["granted"], B, NB)
        torch.add(dev["ctx2"], dev["new"], out=dev["attend"])
        torch.mul(dev["slots"] < 0, (1 << 31) - 1, out=dev["begin"])
        args = (out, q, kc, vc, dev["tables"], dev["attend"], dev["starts"], scale)
        kw = dict(softcap=cap, window=window, key_begin=dev["begin"], max_query_len=longest, max_context_len=width * B)
        if fp8:
            binding.paged_kv_write_fp8(kn, vn, kc, vc, dev["slots"], ks, vs)
            binding.paged_attention_multi_query_scored_fp8(*args, k_scale=ks, v_scale=vs, **kw)
        else:
            binding.paged_kv_write(kn, vn, kc, vc, dev["slots"])
            binding.paged_attention_multi_query_scored(*args, **kw)
        dev["ctx"].copy_(dev["ctx3"])
        dev["nfree"].copy_(dev["nfree3"])

    graph = None
    if graphed:
        step()  # an empty step
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    hist, waits = [dict(k=[], v=[]) for _ in range(S)], 0
    free = NB
    for new, gone in steps:
        n = sum(new)
        hq, hk, hv = (torch.randn((T, h, D), generator=g).to(dt) for h in (H, Hkv, Hkv))
        for dst, src in ((q, hq), (kn, hk), (vn, hv)):
            dst.copy_(src)
        dev["new"].copy_(i32(new))
        dev["gone"].copy_(i32(gone))
        out.fill_(9.0)
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        at, need, granted = 0, 0, []
        for s in range(S):
            if gone[s]:
                free += -(-len(hist[s]["k"]) // B)
                hist[s] = dict(k=[], v=[])
        for s in range(S):
            have = len(hist[s]["k"])
            blocks = -(-(have + new[s]) // B) - -(-have // B)
            need += blocks
            granted.append(int(blocks == 0 or need <= free))
            if granted[s]:
                hist[s]["k"] += list(hk[at:at + new[s]])
                hist[s]["v"] += list(hv[at:at + new[s]])
            at += new[s]
        free = NB - sum(-(-len(h["k"]) // B) for h in hist)
        waits += granted.count(0)
        ctx = [len(h["k"]) for h in hist]
        assert dev["granted"].tolist() == granted and dev["ctx3"].tolist() == ctx and dev["nfree"].item() == free
        # the definition, over the sequences that were granted
        b = R.build(1, ctx, [x if w else 0 for x, w in zip(new, granted)], H, Hkv, D, B, "bf16", fp8)
        if fp8:
            b.update(k_scale=ks, v_scale=vs)
        for s in range(S):
            for j in range(ctx[s]):
                for pool, name, sc in (("kc", "k", ks), ("vc", "v", vs)):
                    x = hist[s][name][j]
                    if fp8:
                        x = (x.float() / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    b[pool][b["tables"][s, j // B], :, j % B] = x
        starts = [sum(new[:s]) for s in range(S + 1)]
        mine = [t for s in range(S) if granted[s] for t in range(starts[s], starts[s + 1])]
        others = [t for t in range(n) if t not in mine]
        b["q"] = hq[mine]
        ref, tol = R.reference(b, softcap=cap, window=window)
        assert R.worst(out[mine], ref, tol) <= 1.0
        assert (out[others] == 0).all() and (out[n:] == 9.0).all()
        assert binding.device_errors() == 0
    assert waits == waiting


def test_bad_tensors_are_refused(cuda_lib):
    """Another type, layout, device or shape of any array raises before anything is launched."""
    def args(**kw):
        S = 3
        a = dict(block_tables=torch.zeros((S, 4), dtype=torch.int32, device=DEV), context_lens=i32([1] * S),
                 new_lens=i32([1] * S), free_blocks=i32([5, 6]), num_free=i32([2]),
                 slot_mapping=torch.zeros(8, dtype=torch.int64, device=DEV), query_start_loc=i32([0] * (S + 1)),
                 context_lens_out=i32([0] * S), num_free_out=i32([0]), granted=i32([0] * S), block_size=16,
                 num_blocks=8)
        a.update(kw)
        return a

    binding.paged_kv_reserve_slots(**args())
    wide = torch.zeros((3, 8), dtype=torch.int32, device=DEV)
    for kw in (dict(context_lens=i32([1, 1, 1]).long()), dict(block_tables=wide[:, ::2]), dict(new_lens=i32([1, 1])),
               dict(slot_mapping=i32([0] * 8)), dict(query_start_loc=i32([0, 0, 0])), dict(granted=i32([0, 0])),
               dict(num_free=i32([1, 2])), dict(free_blocks=torch.zeros(2, dtype=torch.int32)),
               dict(context_lens_out=torch.zeros(3, dtype=torch.int32)), dict(block_size=12),
               dict(block_tables=i32([0] * 12))):
        with pytest.raises(binding.PagedKVError):
            binding.paged_kv_reserve_slots(**args(**kw))
    same = i32([1, 1, 1])
    with pytest.raises(binding.PagedKVError):
        binding.paged_kv_reserve_slots(**args(context_lens=same, context_lens_out=same))
    with pytest.raises(binding.PagedKVError):
        binding.paged_kv_reserve_slots(**args(context_lens=same, granted=same))
