"""The passes around tree attention (layout, accepted rows moved up, blocks trimmed) against their rules in plain Python,
exactly; and serving loops of whole speculative steps."""
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


def starts_of(qlens):
    starts = [0]
    for q in qlens:
        starts.append(starts[-1] + q)
    return starts


# ---- masks and positions


def layout(pars, committed, W=None, pad=0, max_q=None):
    qlens = [len(p) for p in pars]
    W = W or max(1, R.ceil_div(max(qlens + [1]), 32))
    T = sum(qlens) + pad
    mask = torch.full((T, W), 77, dtype=torch.int32, device=DEV)
    positions = torch.full((T,), 77, dtype=torch.int32, device=DEV)
    flat = [x for p in pars for x in p] + [-5] * pad
    binding.paged_kv_tree_layout(i32(flat), i32(starts_of(qlens)), i32([c + q for c, q in zip(committed, qlens)]), mask,
                                 positions, max_query_len=max_q)
    torch.cuda.synchronize()
    return mask.cpu(), positions.tolist()


@pytest.mark.parametrize("shape", ["tree", "chain", "star"])
@pytest.mark.parametrize("qlens,W", [([1], None), ([3, 0, 1, 7], 2), ([31, 32, 33, 64, 65], None),
                                     ([255, 8], 40), ([1024], None), ([20] * 300, None)])
def test_layout(qlens, W, shape):
    committed = [(37 * s) % 1000 for s in range(len(qlens))]
    pars = [TR.parents(s, q, 1 + s % 3, shape) for s, q in enumerate(qlens)]
    mask, positions = layout(pars, committed, W, pad=3)
    sets = [TR.ancestors(p) for p in pars]
    want = TR.words_of([v for x in sets for v in x], mask.shape[1])
    assert torch.equal(mask[:-3], want) and (mask[-3:] == 77).all()
    assert positions == [c + len(v) - 1 for c, x in zip(committed, sets) for v in x] + [77] * 3
    assert binding.device_errors() == 0


def test_layout_reports_bad_parents_and_offsets():
    mask, positions = layout([[-1, 1, 5, 2], [-9, 0]], [10, 20])  # nodes 1 and 2 name no earlier one
    assert mask[:, 0].tolist() == [1, 2, 4, 12, 1, 3] and positions == [10, 10, 10, 11, 20, 21]
    assert binding.device_errors(clear=True) == 16
    mask, positions = layout([[-1, 0], [-1, 0], [-1]], [3, -1, 4])  # the second has more drafted tokens than context
    assert positions == [3, 4, 77, 77, 4] and (mask[2:4] == 77).all()
    assert binding.device_errors(clear=True) == 16
    mask, positions = layout([[-1, 0], [-1, 0, 1], [-1]], [3, 3, 4], max_q=2)
    assert positions == [3, 4, 77, 77, 77, 4]
    assert binding.device_errors(clear=True) == 16


# ---- accepted rows


def pools(g, layers, NB, Hkv, B, D, dtype):
    if dtype == torch.uint8:
        return [torch.randint(0, 256, (layers, NB, Hkv, B, D), generator=g, dtype=dtype) for _ in range(2)]
    return [torch.randn((layers, NB, Hkv, B, D), generator=g).to(dtype) for _ in range(2)]


def tables_of(g, ctx, B, spare=2):
    used = [R.ceil_div(n, B) for n in ctx]
    NB = sum(used) + spare
    perm = torch.randperm(NB, generator=g).tolist()
    t = torch.full((len(ctx), max(used + [1])), -1, dtype=torch.int32)
    for s, n in enumerate(used):
        for j in range(n):
            t[s, j] = perm.pop()
    return t, NB


def moved(pool, tables, committed, paths, B):
    want = pool.clone()
    for s, path in enumerate(paths):
        for i, u in enumerate(path):
            a, b = committed[s] + u, committed[s] + i
            want[:, tables[s, b // B], :, b % B] = want[:, tables[s, a // B], :, a % B].clone()
    return want


def compact(kc, vc, tables, ctx, qlens, paths):
    k, v = kc.to(DEV), vc.to(DEV)
    width = max([1] + [len(p) for p in paths])
    acc = i32([(p + [-1] * width)[:width] for p in paths])
    binding.paged_kv_compact_accepted(k, v, tables.to(DEV), i32(ctx), i32(starts_of(qlens)), acc,
                                      i32([len(p) for p in paths]))
    torch.cuda.synchronize()
    return k.cpu(), v.cpu()


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("layers,Hkv,D,B,dtype", [
    (1, 1, 64, 8, torch.float16), (3, 2, 128, 16, torch.bfloat16), (2, 3, 128, 32, torch.uint8), (1, 2, 64, 16, torch.uint8),
    (9, 8, 64, 16, torch.bfloat16), (7, 5, 128, 8, torch.uint8)])
@pytest.mark.parametrize("qlens", [[1], [5, 0, 16, 3], [64, 33, 200], [400]])
def test_compact(layers, Hkv, D, B, dtype, qlens):
    g = torch.Generator().manual_seed(layers + D + len(qlens))
    r = random.Random(layers * 100 + len(qlens))
    committed = [r.randint(0, 50) for _ in qlens]
    ctx = [c + q for c, q in zip(committed, qlens)]
    tables, NB = tables_of(g, ctx, B)
    kc, vc = pools(g, layers, NB, Hkv, B, D, dtype)
    for share in (0.0, 0.2, 0.7, 1.0):
        paths = [sorted(u for u in range(q) if r.random() < share) for q in qlens]
        k, v = compact(kc, vc, tables, ctx, qlens, paths)
        assert same_bits(k, moved(kc, tables, committed, paths, B)) and same_bits(v, moved(vc, tables, committed, paths, B))
    assert binding.device_errors() == 0


def test_compact_of_one_pool_and_float8():
    g = torch.Generator().manual_seed(3)
    tables, NB = tables_of(g, [30], 16)
    kc, vc = pools(g, 1, NB, 2, 16, 128, torch.uint8)
    k, v = compact(kc[0].view(torch.float8_e4m3fn), vc[0].view(torch.float8_e4m3fn), tables, [30], [20], [[1, 4, 19]])
    assert same_bits(k[None], moved(kc, tables, [10], [[1, 4, 19]], 16)) and not same_bits(v[None], vc)


def test_compact_leaves_bad_sequences():
    g = torch.Generator().manual_seed(4)
    ctx, qlens = [40] * 6, [10] * 6
    tables, NB = tables_of(g, ctx, 16)
    kc, vc = pools(g, 2, NB, 2, 16, 128, torch.bfloat16)
    for bad in ([3, 3], [5, 2], [-1, 4], [2, 10], [1 << 30]):
        paths = [[2, 5], bad, [1], [], [0, 9], [4]]
        k, v = compact(kc, vc, tables, ctx, qlens, paths)
        fine = [p if p is not bad else [] for p in paths]
        assert same_bits(k, moved(kc, tables, [30] * 6, fine, 16)) and same_bits(v, moved(vc, tables, [30] * 6, fine, 16))
        assert binding.device_errors(clear=True) == 16
    # more than the array holds, fewer than none, more context than table, more drafted tokens than context
    for n, c, error in ((3, 40, 16), (-1, 40, 16), (1, 49, 2), (1, 9, 16)):
        k, v = kc.to(DEV), vc.to(DEV)
        binding.paged_kv_compact_accepted(k, v, tables[:1].to(DEV), i32([c]), i32([0, 10]), i32([[3, 4]]), i32([n]))
        torch.cuda.synchronize()
        assert same_bits(k.cpu(), kc) and same_bits(v.cpu(), vc)
        assert binding.device_errors(clear=True) == error
    tables[0, 1], tables[0, 2] = NB, -1  # places 30 .. 39 lie in blocks that are not the pool's
    k, v = compact(kc, vc, tables[:1], [40], [10], [[1, 3]])
    assert same_bits(k, kc) and same_bits(v, vc) and binding.device_errors(clear=True) == 1


def test_compact_over_far_layers():
    """Layers whose pools lie more than 2^31 bytes apart."""
    NB, Hkv, B, D = 5000, 8, 32, 128  # 328 MB a layer
    g = torch.Generator(device=DEV).manual_seed(5)
    kc = torch.zeros((15, NB, Hkv, B, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    tables = i32([[NB - 1, 7, NB - 2]])
    rows = torch.randn((2, 15, Hkv, D), generator=g, device=DEV).to(torch.bfloat16)
    kc[:, NB - 2, :, 5], vc[:, NB - 2, :, 5] = rows[0], rows[1]  # place 69
    binding.paged_kv_compact_accepted(kc, vc, tables, i32([80]), i32([0, 60]), i32([[49]]), i32([1]))
    torch.cuda.synchronize()
    assert torch.equal(kc[:, NB - 1, :, 20], rows[0]) and torch.equal(vc[:, NB - 1, :, 20], rows[1])
    assert binding.device_errors() == 0


# ---- trimmed blocks


def trim(tables, ctx, keep, stack, nfree, B, NB):
    stack, ctx_out, free_out = i32(stack), i32([-5] * len(ctx)), i32([-5])
    t = i32(tables).reshape(len(ctx), -1) if ctx else torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    binding.paged_kv_trim_blocks(t, i32(ctx), i32(keep), stack, i32([nfree]), ctx_out, free_out, B, NB)
    torch.cuda.synchronize()
    return stack.tolist(), ctx_out.tolist(), free_out.tolist()


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("S,hi,drop", [(0, 1, 1), (1, 40, 3), (5, 300, 300), (64, 300, 20), (303, 90, 30), (2049, 64, 64),
                                       (5000, 40, 9)])
def test_trim(S, hi, drop, B):
    r = random.Random(S + hi + B)
    ctx = [r.randint(0, hi) for _ in range(S)]
    keep = [r.choice([n, max(0, n - r.randint(0, drop)), 0]) for n in ctx]
    used = [R.ceil_div(n, B) for n in ctx]
    NB = sum(used) + 4
    ids = list(range(NB))
    r.shuffle(ids)
    width = max([1] + used)
    tables = [[ids.pop() for _ in range(n)] + [-1] * (width - n) for n in used]
    stack = ids + [-2] * (NB - len(ids))
    want, n = list(stack), len(ids)
    for s in range(S):
        for j in range(R.ceil_div(keep[s], B), used[s]):
            want[n] = tables[s][j]
            n += 1
    assert trim(tables, ctx, keep, stack, len(ids), B, NB) == (want, keep, [n])
    assert binding.device_errors() == 0


def test_trim_reports_bad_lengths():
    tables, stack = [[0, 1, 2], [3, 4, 5], [6, 7, 8]], [-2] * 9
    got = trim(tables, [40, 40, 40], [41, -1, 20], stack, 0, 16, 9)  # keeps 40, 0 and 20
    assert got == ([3, 4, 5, 8] + [-2] * 5, [40, 0, 20], [4])
    assert binding.device_errors(clear=True) == 2
    got = trim(tables, [60, -3, 40], [17, 0, 40], stack, 0, 16, 9)  # contexts of 48 and 0
    assert got == ([2] + [-2] * 8, [17, 0, 40], [1])
    assert binding.device_errors(clear=True) == 2
    got = trim([[0, 99, 2]], [48], [1], [5, -2], 1, 16, 9)  # a block that is none, and a stack that is too small
    assert got == ([5, -1], [1], [2])
    assert binding.device_errors(clear=True) == 1


# ---- whole steps


def turn_table(most, D):
    a = torch.arange(most, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2).double() / D)
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


class Server:
    """Sequences of drafted steps over GPU block tables, beside each sequence's committed rows on the host."""

    def __init__(self, seed, S, H, Hkv, D, B, fp8, NB, layers=2, width=30):
        self.r, self.g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.S, self.H, self.Hkv, self.D, self.B, self.fp8, self.NB, self.layers = S, H, Hkv, D, B, fp8, NB, layers
        self.dtype = torch.bfloat16
        shape = (layers, NB, Hkv, B, D)
        bad = 0x7F if fp8 else float("nan")
        self.kc, self.vc = (torch.full(shape, bad, dtype=torch.uint8 if fp8 else self.dtype, device=DEV) for _ in range(2))
        self.tables = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
        self.ctx, self.free = i32([0] * S), torch.randperm(NB, generator=self.g).to(torch.int32).to(DEV)
        self.num_free = i32([NB])
        self.committed = [0] * S
        self.rows = [[None] * S for _ in range(layers)]  # committed K and V values, [n][Hkv][D] float64
        self.cs = turn_table(400, D)
        self.w = (1 + 0.2 * torch.randn(D, generator=self.g)).to(DEV)
        self.scales = (0.02, 0.02) if fp8 else ()

    def stored(self, pool, layer, s, places):
        p = torch.tensor(list(places), dtype=torch.long)
        x = pool[layer].cpu()[self.tables[s].cpu()[p // self.B].long(), :, p % self.B]
        return x.view(torch.float8_e4m3fn).double() * 0.02 if self.fp8 else x.double()

    def step(self, qlens, expect_wait=()):
        S, H, Hkv, D, B = self.S, self.H, self.Hkv, self.D, self.B
        T, starts = sum(qlens), starts_of(qlens)
        pars = [TR.parents(self.r.random(), q, self.r.randint(1, 2)) for q in qlens]
        sets = [TR.ancestors(p) for p in pars]
        slots = torch.empty(T + 3, dtype=torch.int64, device=DEV)
        qsl, ctx2, free2, granted = i32([0] * (S + 1)), i32([0] * S), i32([0]), i32([0] * S)
        new = i32(qlens)
        binding.paged_kv_reserve_slots(self.tables, self.ctx, new, self.free, self.num_free, slots, qsl, ctx2, free2,
                                       granted, B, self.NB)
        attend = self.ctx + new
        begin = (slots[:T] < 0).to(torch.int32) * HIDE
        W = R.ceil_div(max(qlens), 32)
        mask, pos = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((T, W), (T,)))
        binding.paged_kv_tree_layout(i32([x for p in pars for x in p]), qsl, attend, mask, pos, max_query_len=max(qlens))
        outs, qs = [], []
        for layer in range(self.layers):
            qkv = torch.randn((T, H + 2 * Hkv, D), generator=self.g).to(self.dtype).to(DEV)
            q = torch.empty((T, H, D), dtype=self.dtype, device=DEV)
            f = "_fp8" if self.fp8 else ""
            getattr(binding, "paged_kv_write_rope" + f)(
                q, qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], self.kc[layer], self.vc[layer], slots[:T], pos, self.cs,
                *self.scales, q_weight=self.w, k_weight=self.w)
            out = torch.full_like(q, float("nan"))
            getattr(binding, "paged_attention_tree" + f)(
                out, q, self.kc[layer], self.vc[layer], self.tables, attend, qsl, mask, D ** -0.5, *self.scales,
                key_begin=begin, max_query_len=max(qlens))
            outs.append(out)
            qs.append(q)
        wait = [s for s in range(S) if not granted[s].item()]
        assert tuple(wait) == tuple(expect_wait)
        paths = [sorted(self.r.choice(x)) if x and s not in wait and self.r.random() < 0.9 else []
                 for s, x in enumerate(sets)]
        # what the step computed, before the rows move
        for layer in range(self.layers):
            b = dict(H=H, Hkv=Hkv, D=D, B=B, kc=self.kc[layer].cpu(), vc=self.vc[layer].cpu(), k_scale=0.02, v_scale=0.02,
                     fp8=self.fp8, dtype=self.dtype, q=qs[layer].cpu(), committed=self.committed, qlens=qlens,
                     starts=starts, scale=D ** -0.5, tables=self.tables.cpu(), sets=[v for x in sets for v in x])
            ref, tol = TR.reference(b, key_begin=begin.tolist())
            assert R.worst(outs[layer], ref, tol) <= 1.0
            for s in range(S):  # the committed rows are where and what they were
                if self.committed[s]:
                    for pool, was in zip((self.kc, self.vc), self.rows[layer][s]):
                        assert torch.equal(self.stored(pool, layer, s, range(self.committed[s])), was)
        want = [[[self.stored(pool, layer, s, list(range(self.committed[s])) + [self.committed[s] + u for u in paths[s]])
                  for pool in (self.kc, self.vc)] for s in range(S)] for layer in range(self.layers)]
        width = max([1] + [len(p) for p in paths])
        num = i32([len(p) for p in paths])
        binding.paged_kv_compact_accepted(self.kc, self.vc, self.tables, attend, qsl,
                                          i32([p + [-1] * (width - len(p)) for p in paths]), num)
        keep, ctx3, free3 = self.ctx + num, i32([0] * S), i32([0])
        binding.paged_kv_trim_blocks(self.tables, ctx2, keep, self.free, free2, ctx3, free3, B, self.NB)
        self.ctx, self.num_free, self.rows = ctx3, free3, want
        self.committed = [c + len(p) for c, p in zip(self.committed, paths)]
        assert self.ctx.tolist() == self.committed
        used = [self.tables[s, :R.ceil_div(c, B)].tolist() for s, c in enumerate(self.committed)]
        ids = [x for u in used for x in u] + self.free[:self.num_free.item()].tolist()
        assert sorted(ids) == list(range(self.NB))  # every block has one owner
        assert binding.device_errors() == 0


@pytest.mark.parametrize("H,Hkv,D,B,fp8", [(8, 2, 128, 16, False), (4, 4, 64, 8, False), (8, 1, 128, 16, True)])
def test_speculative_steps(H, Hkv, D, B, fp8):
    server = Server(51, 5, H, Hkv, D, B, fp8, NB=90)
    for k in range(6):
        server.step([server.r.choice([1, 4, 9, 40]) if k else 30 for _ in range(5)])


def test_speculative_steps_with_sequences_that_wait():
    server = Server(52, 3, 4, 2, 128, 16, False, NB=5, layers=1)
    server.step([20, 30, 40], expect_wait=[2])  # 2 + 2 blocks, the third wants 3
    server.step([3, 3, 3])


def test_a_captured_step():
    """Layout, write, attention, compaction and trimming in one graph, replayed with other trees in its buffers."""
    S, H, Hkv, D, B, q = 3, 8, 2, 128, 16, 12
    batches = [TR.build(60 + k, [50, 3, 120], [q] * S, H, Hkv, D, B) for k in range(3)]
    b = batches[0]
    NB, T = b["kc"].shape[0], S * q
    r = random.Random(8)
    dev = {k: b[k].to(DEV) for k in ("q", "kc", "vc", "tables")}
    g = torch.Generator().manual_seed(9)
    k_new, v_new = (torch.randn((T, Hkv, D), generator=g).to(b["dtype"]).to(DEV) for _ in range(2))
    ctx, qsl = i32(b["ctx"]), i32(b["starts"])
    par, acc, num = i32([-1] * T), i32([[0] * q] * S), i32([0] * S)
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    mask, pos = torch.empty((T, 1), dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV)
    stack, nfree = torch.full((NB,), -1, dtype=torch.int32, device=DEV), i32([0])
    ctx_out, free_out, out, q_out = i32([0] * S), i32([0]), torch.empty_like(dev["q"]), torch.empty_like(dev["q"])
    cs = turn_table(300, D)
    need = binding.paged_attention_tree_workspace_size(T, H, Hkv, D, B, q, max(b["ctx"]))
    ws = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)

    def step():
        binding.paged_kv_tree_layout(par, qsl, ctx, mask, pos, max_query_len=q)
        binding.paged_kv_write_rope(q_out, dev["q"], k_new, v_new, dev["kc"], dev["vc"], slots, pos, cs)
        binding.paged_attention_tree(out, q_out, dev["kc"], dev["vc"], dev["tables"], ctx, qsl, mask, b["scale"],
                                     max_query_len=q, max_context_len=max(b["ctx"]), workspace=ws)
        binding.paged_kv_compact_accepted(dev["kc"], dev["vc"], dev["tables"], ctx, qsl, acc, num)
        binding.paged_kv_trim_blocks(dev["tables"], ctx, ctx - q + num, stack, nfree, ctx_out, free_out, B, NB)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in batches[1:]:
        sets = [TR.ancestors(p) for p in x["parents"]]
        paths = [sorted(r.choice(v)) for v in sets]
        for k in ("q", "kc", "vc", "tables"):
            dev[k].copy_(x[k])
        par.copy_(i32([y for p in x["parents"] for y in p]))
        acc.copy_(i32([p + [-1] * (q - len(p)) for p in paths]))
        num.copy_(i32([len(p) for p in paths]))
        places = [(s, c + u) for s, c in enumerate(x["committed"]) for u in range(q)]
        slots.copy_(torch.tensor([int(x["tables"][s, p // B]) * B + p % B for s, p in places]))
        graph.replay()
        torch.cuda.synchronize()
        # the state before compaction: the replayed write's rows, which the call gives again on the same inputs
        kc, vc, q2 = x["kc"].to(DEV), x["vc"].to(DEV), torch.empty_like(q_out)
        binding.paged_kv_write_rope(q2, dev["q"], k_new, v_new, kc, vc, slots, pos, cs)
        ref, tol = TR.reference(dict(x, q=q2.cpu(), kc=kc.cpu(), vc=vc.cpu()))
        assert torch.equal(q2, q_out) and R.worst(out, ref, tol) <= 1.0
        for pool, was in ((dev["kc"], kc), (dev["vc"], vc)):
            assert same_bits(pool.cpu()[None], moved(was.cpu()[None], x["tables"], x["committed"], paths, B))
        keep = [c + len(p) for c, p in zip(x["committed"], paths)]
        assert ctx_out.tolist() == keep
        want = [int(x["tables"][s, j]) for s in range(S) for j in range(R.ceil_div(keep[s], B), R.ceil_div(x["ctx"][s], B))]
        assert stack[:free_out.item()].tolist() == want
        assert binding.device_errors() == 0
