"""Scored paged attention (tanh cap, distance bias, window, key intervals) on the GPU against the definition in
64 bits, within the error that the formats allow (tests/scored_reference.py)."""
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


def call(b, softcap=0.0, slopes=None, window=0, key_begin=None, key_end=None, out=None, max_ctx=None, **kw):
    out = torch.full_like(b["q"], float("nan"), device=DEV) if out is None else out
    args = [out, b["q"].to(DEV), b["kc"].to(DEV), b["vc"].to(DEV), b["tables"].to(DEV), i32(b["ctx"])]
    kw = dict(kw, softcap=softcap, window=window, alibi_slopes=None if slopes is None else slopes.to(DEV),
              key_begin=None if key_begin is None else i32(key_begin),
              max_context_len=max(b["ctx"]) if max_ctx is None else max_ctx)
    if b["fp8"]:
        kw.update(k_scale=b["k_scale"], v_scale=b["v_scale"])
    if b["decode"]:
        fn = binding.paged_attention_decode_scored_fp8 if b["fp8"] else binding.paged_attention_decode_scored
        fn(*args, b["scale"], **kw)
    else:
        fn = binding.paged_attention_multi_query_scored_fp8 if b["fp8"] else binding.paged_attention_multi_query_scored
        kw.setdefault("max_query_len", max(b["qlens"]))
        fn(*args, i32(b["starts"]), b["scale"], key_end=None if key_end is None else i32(key_end), **kw)
    torch.cuda.synchronize()
    return out


def check(b, errors=0, part=0, **rules):
    ref, tol = R.reference(b, **rules)
    out = call(b, partition_size=part, **rules)
    assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == errors


DECODE_CTX = [0, 1, 7, 8, 9, 31, 33, 64, 65, 200, 300, 511, 777]
SHAPES = [  # H, Hkv, D, B, dtype, fp8
    (4, 4, 64, 16, "f16", False), (8, 2, 128, 16, "bf16", False), (6, 2, 64, 8, "bf16", False),
    (8, 8, 128, 32, "f16", False), (16, 1, 128, 8, "f16", False), (20, 4, 128, 16, "bf16", False),
    (8, 1, 128, 16, "bf16", True), (4, 4, 128, 8, "f16", True), (24, 2, 128, 32, "bf16", True),
    (20, 1, 128, 16, "f16", False), (33, 1, 64, 8, "bf16", False), (40, 2, 128, 32, "bf16", True),
]
RULES = ["none", "cap", "alibi", "window", "begin", "all"]


def rules_of(name, b, seed=5):
    r = {}
    if name in ("cap", "all"):
        r["softcap"] = 3.0  # the scores' spread is about 2: both sides of the tanh's bend
    if name in ("alibi", "all"):
        r["slopes"] = R.slopes_of(b["H"])
    if name in ("window", "all"):
        r["window"] = 70
    if name in ("begin", "all"):
        r["key_begin"] = R.documents(b, seed)
    return r


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", SHAPES)
def test_decode(H, Hkv, D, B, dtype, fp8, rule):
    b = R.build(11, DECODE_CTX, None, H, Hkv, D, B, dtype, fp8)
    check(b, **rules_of(rule, b))


@pytest.mark.parametrize("rule", ["cap", "window", "all"])
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [SHAPES[1], SHAPES[3], SHAPES[5], SHAPES[6]])
def test_decode_split(H, Hkv, D, B, dtype, fp8, rule):
    """Contexts of several partitions (64 tokens each), and a context length bound above them all."""
    b = R.build(12, [1, 64, 65, 129, 640, 901], None, H, Hkv, D, B, dtype, fp8)
    check(b, part=64, **rules_of(rule, b))
    ref, tol = R.reference(b, **rules_of(rule, b))
    out = call(b, partition_size=64, max_ctx=b["tables"].shape[1] * B, **rules_of(rule, b))
    assert R.worst(out, ref, tol) <= 1.0


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 1 << 30])
def test_decode_windows(window):
    b = R.build(13, [1, 2, 15, 16, 17, 100, 500], None, 8, 2, 128, 16)
    check(b, window=window)


@pytest.mark.parametrize("softcap", [1e-3, 0.5, 50.0, 1e6])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_caps(softcap, dtype):
    """Far into the cap, and caps that no score comes near."""
    b = R.build(14, [3, 90, 400], None, 8, 2, 128, 16, dtype, spread=4.0)
    check(b, softcap=softcap)


@pytest.mark.parametrize("softcap", [1e-3, 0.5, 50.0, 1e6])
@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("bf16", True)])
def test_multi_query_caps(softcap, dtype, fp8):
    b = R.build(15, [70, 300, 9], [70, 130, 2], 8, 2, 128, 16, dtype, fp8, spread=4.0)
    check(b, softcap=softcap)
    check(b, softcap=softcap, window=40, key_begin=R.documents(b, 4))


MQ = [  # contexts, query lengths
    ([5, 40, 131, 300], [5, 4, 131, 64]),       # whole prompts and chunks
    ([1, 77, 200, 64, 9], [1, 0, 3, 64, 2]),    # one token, none, few
    ([700], [150]),
]
MQ_RULES = ["none", "cap", "alibi", "window", "documents", "prefix", "full", "all"]


def mq_rules(name, b):
    r = {}
    if name in ("cap", "all"):
        r["softcap"] = 3.0
    if name in ("alibi", "all"):
        r["slopes"] = R.slopes_of(b["H"])
    if name in ("window", "all"):
        r["window"] = 50
    if name == "documents":
        r["key_begin"] = R.documents(b, 8)
    if name in ("prefix", "all"):
        r["key_end"] = R.prefixes(b, 9)
    if name == "full":  # no causal mask, distances on both sides
        r["key_end"] = [1 << 30] * b["q"].shape[0]
        r["slopes"] = R.slopes_of(b["H"])
    return r


@pytest.mark.parametrize("rule", MQ_RULES)
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", SHAPES)
def test_multi_query(H, Hkv, D, B, dtype, fp8, rule):
    for ctx, qlens in MQ[:2]:
        b = R.build(21, ctx, qlens, H, Hkv, D, B, dtype, fp8)
        check(b, **mq_rules(rule, b))


@pytest.mark.parametrize("rule", ["cap", "window", "documents", "prefix", "all"])
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [SHAPES[0], SHAPES[1], SHAPES[5], SHAPES[6]])
def test_multi_query_split(H, Hkv, D, B, dtype, fp8, rule):
    b = R.build(22, *MQ[2], H, Hkv, D, B, dtype, fp8)
    check(b, part=128, **mq_rules(rule, b))


@pytest.mark.parametrize("q", [1, 3, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_see_nothing(q, fp8):
    """Empty intervals, among rows that see something and all through a sequence, give zeros; values far
    outside the context are clamped."""
    b = R.build(23, [60, 200], [q, q], 8, 2, 128, 16, fp8=fp8)
    T = 2 * q
    begin = [(1 << 31) - 1 if t % 3 == 0 else -(1 << 31) for t in range(T)]
    end = [(1 << 31) - 1 if t % 2 else 30 for t in range(T)]
    check(b, key_begin=begin, key_end=end, softcap=2.0)
    check(b, key_begin=[0] * T, key_end=[-(1 << 31)] * T)
    check(b, key_begin=[100] * T, key_end=[100] * T, window=5, slopes=R.slopes_of(8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_decode_masked_keys_may_hold_anything(what, fp8):
    if fp8 and what == "inf":
        pytest.skip("E4M3 has no infinity")
    b = R.build(24, [40, 300, 90], None, 8, 2, 128, 16, fp8=fp8)
    begin = [3, 250, 89]
    bad = 0x7F if fp8 else float(what)
    for s, lo in enumerate(begin):
        for j in range(lo):
            for pool in (b["kc"], b["vc"]):
                pool[b["tables"][s, j // 16], :, j % 16] = bad
    check(b, key_begin=begin, softcap=5.0)
    check(b, key_begin=begin, slopes=R.slopes_of(8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[2, 3], [60, 90]])
@pytest.mark.parametrize("part", [0, 64])
def test_a_key_of_others_never_reaches_a_row(qlens, fp8, part):
    """NaN and infinities in keys that some rows see do not reach the rows that do not see them."""
    b = R.build(25, [100, 200], qlens, 4, 2, 128, 16, "bf16", fp8)
    T = sum(qlens)
    rows = {}
    for s, at in ((0, 97), (1, 150)):  # two keys of NaN values; the second sequence's rows all see past it
        for pool in (b["kc"], b["vc"]):
            pool[b["tables"][s, at // 16], :, at % 16] = 0x7F if fp8 else float("nan")
        rows[s] = at
    if not fp8:
        b["vc"][b["tables"][1, 10], :, 3] = float("inf")
    begin, end = [], []
    for s, (n, ql) in enumerate(zip(b["ctx"], b["qlens"])):
        for i in range(ql):
            sees = i % 2 == 1
            begin.append(0 if sees else rows[s] + 1 if s else 0)
            end.append(n if sees else n if s else rows[s])
    ref, tol = R.reference(b, key_begin=begin, key_end=end, softcap=4.0)
    out = call(b, key_begin=begin, key_end=end, softcap=4.0, partition_size=part).double().cpu()
    clean = [t for t in range(T) if torch.isfinite(ref[t]).all()]
    assert clean and len(clean) < T
    assert R.worst(out[clean], ref[clean], tol[clean]) <= 1.0
    for t in range(T):
        if t not in clean:
            assert not torch.isfinite(out[t]).all()


@pytest.mark.parametrize("qlens", [None, [4, 2], [70, 40]])
def test_blocks_behind_the_window_are_not_read(qlens):
    """Their table entries may be anything: no error is reported."""
    b = R.build(26, [300, 150], qlens, 8, 2, 128, 16)
    ref, tol = R.reference(b, window=20)
    for s, (n, ql) in enumerate(zip(b["ctx"], b["qlens"])):
        b["tables"][s, :(n - ql - 20 + 1) // 16] = -9 if s else 1 << 30
    out = call(b, window=20)
    assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == 0


@pytest.mark.parametrize("qlens", [None, [5, 3], [60, 90]])
def test_bad_block_ids_are_skipped_and_reported(qlens):
    b = R.build(27, [100, 200], qlens, 8, 2, 128, 16, fp8=False)
    b["tables"][0, 1] = b["kc"].shape[0]
    b["tables"][1, 4] = -1
    check(b, errors=1, softcap=4.0, slopes=R.slopes_of(8))


def test_contexts_are_clamped_and_reported():
    b = R.build(28, [40, 90], None, 4, 2, 64, 16)
    bad = dict(b, ctx=[-3, 400])
    out = call(bad, max_ctx=90, softcap=5.0)
    ref, tol = R.reference(b, softcap=5.0)
    assert R.worst(out[1:], ref[1:], tol[1:]) <= 1.0
    assert (out[0] == 0).all()
    assert binding.device_errors() == 2


@pytest.mark.parametrize("q", [3, 50])
def test_bad_query_offsets_skip_their_sequence(q):
    b = R.build(29, [60, 70, 80], [q, q, q], 8, 2, 128, 16)
    ref, tol = R.reference(b, softcap=5.0)
    for starts, good in (([0, q, q - 1, 3 * q], [0]), ([0, q, 2 * q, 3 * q + 1], [0, 1]),
                         ([-1, q, 2 * q, 3 * q], [1, 2])):
        # ([0, q, q - 1, 3q]: sequence 1 has a negative length, sequence 2 more tokens than max_query_len)
        out = call(dict(b, starts=starts), softcap=5.0)
        for s in range(3):
            rows = slice(s * q, (s + 1) * q)
            if s in good:
                assert R.worst(out[rows], ref[rows], tol[rows]) <= 1.0
            else:
                assert torch.isnan(out[rows]).all()
        assert binding.device_errors() == 16


def test_rows_past_the_last_sequence_are_left_as_they_were():
    b = R.build(30, [50, 90], [20, 30], 8, 2, 128, 16)
    ref, tol = R.reference(b, window=33)
    big = dict(b, q=torch.cat([b["q"], b["q"][:7]]))
    out = torch.full_like(big["q"], 7.5, device=DEV)
    call(big, window=33, out=out)
    assert R.worst(out[:50], ref, tol) <= 1.0
    assert (out[50:] == 7.5).all()


@pytest.mark.parametrize("qlens", [None, [4, 9], [80, 33]])
def test_other_stream_and_graph(qlens):
    """On another stream, and captured once and replayed over new inputs."""
    rules = dict(softcap=4.0, window=60, slopes=R.slopes_of(8))
    one, two = (R.build(seed, [200, 170], qlens, 8, 2, 128, 16) for seed in (31, 32))
    want = [R.reference(x, **rules) for x in (one, two)]
    st = {k: one[k].to(DEV) for k in ("q", "kc", "vc", "tables")}
    out = torch.empty_like(st["q"])
    ctx, starts, slopes = i32(one["ctx"]), i32(one["starts"]), rules["slopes"].to(DEV)
    mql = max(one["qlens"])
    need = binding.paged_attention_scored_workspace_size(st["q"].shape[0], 8, 2, 128, 16, mql, 200, 60, 64)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        a = (out, st["q"], st["kc"], st["vc"], st["tables"], ctx)
        kw = dict(softcap=4.0, window=60, alibi_slopes=slopes, max_context_len=200, partition_size=64, workspace=ws,
                  stream=stream)
        if qlens is None:
            binding.paged_attention_decode_scored(*a, one["scale"], **kw)
        else:
            binding.paged_attention_multi_query_scored(*a, starts, one["scale"], max_query_len=mql, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    assert R.worst(out, *want[0]) <= 1.0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in ("q", "kc", "vc", "tables"):
        st[k].copy_(two[k])
    for _ in range(2):
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert R.worst(out, *want[1]) <= 1.0


@pytest.mark.parametrize("qlens", [None, [70, 90]])
def test_same_inputs_give_the_same_bits(qlens):
    b = R.build(33, [333, 500], qlens, 8, 2, 128, 16)
    first = call(b, softcap=9.0, partition_size=64)
    for _ in range(3):
        assert torch.equal(call(b, softcap=9.0, partition_size=64), first)


@pytest.mark.parametrize("qlens", [None, [3, 4], [70, 90]])
def test_bad_tensors_are_refused(qlens):
    """Another type, layout, device or shape of any tensor raises before anything is launched."""
    b = R.build(34, [100, 150], qlens, 4, 2, 64, 16)
    T = b["q"].shape[0]
    q, kc, vc, bt = (b[k].to(DEV) for k in ("q", "kc", "vc", "tables"))
    ok = dict(out=torch.empty_like(q), query=q, key_cache=kc, value_cache=vc, block_tables=bt,
              context_lens=i32(b["ctx"]), scale=0.125, max_context_len=150)
    fn = binding.paged_attention_decode_scored
    if qlens is not None:
        fn = binding.paged_attention_multi_query_scored
        ok.update(query_start_loc=i32(b["starts"]), max_query_len=max(qlens))
    fn(**ok)
    bad = [dict(out=torch.empty_like(q).half()), dict(key_cache=kc.half()), dict(value_cache=vc[:-1]),
           dict(query=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(query=q.cpu()),
           dict(out=torch.empty_like(q[:-1])),
           dict(block_tables=bt.long()), dict(block_tables=bt[:1]), dict(context_lens=i32([1])),
           dict(alibi_slopes=torch.ones(3, device=DEV)), dict(alibi_slopes=torch.ones(4, device=DEV).double()),
           dict(key_begin=i32([0] * (T + 1))), dict(key_begin=torch.zeros(T, device=DEV)), dict(softcap=-1.0),
           dict(window=-1), dict(partition_size=24), dict(max_context_len=10 ** 6),
           dict(partition_size=16, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
           dict(partition_size=16, workspace=torch.empty(1 << 20, dtype=torch.uint8))]
    if qlens is not None:
        bad += [dict(key_end=i32([0] * (T - 1))), dict(query_start_loc=i32([0, T])), dict(max_query_len=151)]
    for kw in bad:
        with pytest.raises(binding.PagedKVError):
            fn(**{**ok, **kw})
    torch.cuda.synchronize()
    assert binding.device_errors() == 0


@pytest.mark.parametrize("qlens", [None, [70, 90]])
def test_workspace_of_a_call_on_another_stream(qlens):
    """A call on a side stream with a workspace of its own making, beside work on the current stream."""
    b = R.build(35, [900, 700], qlens, 8, 2, 128, 16)
    ref, tol = R.reference(b, softcap=6.0)
    side = torch.cuda.Stream()
    out = torch.full_like(b["q"], float("nan"), device=DEV)
    torch.cuda.synchronize()
    for _ in range(4):
        junk = [torch.full((1 << 18,), float("nan"), device=DEV) for _ in range(4)]
        call(b, softcap=6.0, partition_size=64, stream=side, out=out)
        del junk
    assert R.worst(out, ref, tol) <= 1.0


def test_two_calls_at_once():
    """Calls of every tile on two streams at a time give what they give alone."""
    cases = [(R.build(36, [700, 90, 300], None, 8, 2, 128, 16), dict(window=200)),
             (R.build(37, [300, 400], [130, 60], 8, 2, 128, 16), dict(softcap=4.0)),
             (R.build(38, [300, 400], [130, 60], 8, 2, 128, 16, fp8=True), dict(slopes=R.slopes_of(8)))]
    alone = [call(b, partition_size=128, **r) for b, r in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.full_like(b["q"], float("nan"), device=DEV) for b, _ in cases]
    kept = []
    for _ in range(3):
        for (b, r), s, o in zip(cases, streams, outs):
            t = [x.to(DEV) for x in (b["q"], b["kc"], b["vc"], b["tables"])] + [i32(b["ctx"]), i32(b["starts"])]
            sl = r["slopes"].to(DEV) if "slopes" in r else None
            kept += t + [sl]
            torch.cuda.synchronize()
            kw = dict(softcap=r.get("softcap", 0.0), window=r.get("window", 0), alibi_slopes=sl, partition_size=128,
                      max_context_len=max(b["ctx"]), stream=s)
            if b["decode"]:
                binding.paged_attention_decode_scored(o, *t[:5], b["scale"], **kw)
            elif b["fp8"]:
                binding.paged_attention_multi_query_scored_fp8(o, *t[:5], t[5], b["scale"], b["k_scale"], b["v_scale"],
                                                               max_query_len=130, **kw)
            else:
                binding.paged_attention_multi_query_scored(o, *t[:5], t[5], b["scale"], max_query_len=130, **kw)
    torch.cuda.synchronize()
    for o, a in zip(outs, alone):
        assert torch.equal(o, a)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_work_items(fp8):
    """More row tiles than SMs, of very different lengths, empty ones among them: a CTA takes one after the other."""
    ctx = [40 * (i % 11) + 3 for i in range(90)]
    qlens = [0 if i % 7 == 3 else min(n, 1 + 37 * (i % 5)) for i, n in enumerate(ctx)]
    b = R.build(39, ctx, qlens, 16, 4, 128, 16, "bf16", fp8)
    T = sum(qlens)
    begin = [(t * 37) % 90 if t % 13 else 1 << 20 for t in range(T)]
    check(b, key_begin=begin, softcap=3.0)
    check(b, window=25, slopes=R.slopes_of(16), part=64)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("where", [[5], [5, 700], [300, 301]])
def test_a_nan_in_a_long_prompt(where, fp8):
    """A NaN value row reaches the tokens that see it, from its position on, and no earlier one."""
    n = 800
    b = R.build(40, [n], [n], 4, 1, 128, 16, "bf16", fp8)
    for j in where:
        b["vc"][b["tables"][0, j // 16], :, j % 16] = 0x7F if fp8 else float("nan")
    out = call(b, softcap=5.0).double().cpu()
    clean = dict(b, qlens=[where[0]], ctx=[where[0]], q=b["q"][:where[0]])
    ref, tol = R.reference(clean, softcap=5.0)
    assert R.worst(out[:where[0]], ref, tol) <= 1.0
    assert torch.isnan(out[where[0]:]).all()


def test_one_bad_value_in_many_tiles_costs_little():
    """4096 tokens that all see a NaN key keep to the tile: no row is computed again for a value that is its own."""
    n, H, Hkv, D, B = 4096, 16, 4, 128, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    kc, vc = (torch.randn((n // B, Hkv, B, D), device=DEV, dtype=torch.bfloat16, generator=g) for _ in range(2))
    q = torch.randn((n, H, D), device=DEV, dtype=torch.bfloat16, generator=g)
    tables = torch.arange(n // B, device=DEV, dtype=torch.int32)[None].contiguous()
    out = torch.empty_like(q)
    times = []
    for bad in (False, True):
        if bad:
            vc[0, :, 0] = float("nan")
        for _ in range(2):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            binding.paged_attention_multi_query_scored(out, q, kc, vc, tables, i32([n]), i32([0, n]), 0.1, softcap=9.0,
                                                       max_query_len=n, max_context_len=n)
            end.record()
            torch.cuda.synchronize()
        times.append(start.elapsed_time(end))
    assert torch.isnan(out).all()
    assert times[1] < 100 * times[0] + 50.0  # (key by key it would be thousands of times)


def test_a_workspace_for_more_fits_less():
    """A workspace sized for a larger batch serves every smaller one, however that is split."""
    kw = dict(num_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_query_len=1, max_context_len=6000)
    big = binding.paged_attention_scored_workspace_size(7, **kw)
    ws = torch.empty(max(big, 16), dtype=torch.uint8, device=DEV)
    for S in range(1, 8):
        b = R.build(41 + S, [6000 - 777 * i for i in range(S)], None, 8, 2, 128, 16)
        ref, tol = R.reference(b, softcap=5.0)
        out = call(b, softcap=5.0, workspace=ws, max_ctx=6000)
        assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == 0


@pytest.mark.parametrize("H,Hkv,D,dtype", [(16, 1, 128, "bf16"), (16, 2, 64, "f16")])
def test_rows_shared_by_the_streams_after_a_short_item(H, Hkv, D, dtype):
    """Row tiles of more than 128 rows and one tile of keys, first of their CTA, and then row tiles of few rows and
    many keys: the second stream may reach the latter before the first stream's queries of the former are there."""
    G = H // Hkv
    first, then = 320 // Hkv, 320 // Hkv  # more than two items an SM
    q_len = [-(-(129 + 13 * (i % 9)) // G) for i in range(first)] + [1 + i % (128 // G) for i in range(then)]
    q_len[-1] = 256 // G  # (row tiles of 256 rows for the batch)
    ctx = [max(q_len[i], 20 + i % 90) for i in range(first)] + [140 + 50 * (i % 7) for i in range(then)]
    b = R.build(60, ctx, q_len, H, Hkv, D, 16, dtype)
    ref, tol = R.reference(b, softcap=5.0)
    outs = [call(b, softcap=5.0) for _ in range(8)]
    assert R.worst(outs[0], ref, tol) <= 1.0
    assert all(torch.equal(o, outs[0]) for o in outs)
    assert binding.device_errors() == 0


@pytest.mark.parametrize("qlens", [None, [2], [40]])
@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("f16", True)])
def test_a_score_beyond_half_the_cap_leaves_the_others_alone(dtype, fp8, qlens):
    """A cap far above most scores, and a query head whose scores reach it, beside heads with ordinary ones in the same
    tile: each score is as exact as it would be alone."""
    b = R.build(62, [13 if qlens is None else qlens[0] + 12], qlens, 8, 1, 128, 16, dtype, fp8)
    cap = 3e5
    phys = b["tables"][0, 0]
    key = R.values(b, b["kc"], b["k_scale"])[phys, 0, 5]
    b["q"][:, 3] = (6e4 * key.sign()).to(b["dtype"])
    assert (b["q"][0, 3].double() @ key) * b["scale"] > 0.6 * cap
    ref, tol = R.reference(b, softcap=cap)
    out = call(b, softcap=cap)
    rest = [h for h in range(8) if h != 3]
    assert R.worst(out[:, rest], ref[:, rest], tol[:, rest]) <= 1.0
    assert R.worst(out, ref, tol) <= 1.0


def capped_pair(cap, dtype, fp8, z):
    """Two tiles of keys, of which two score z times the cap for every query, with values 1 and -1, so that each row is
    0; beside the second one stands a key beyond half the cap, which leaves its half of the tile to the exponential
    form of the tanh, while the first one's takes the polynomial. A score off by d in one of them moves a row by d / 2."""
    n, ql, H, D = 256, 40, 8, 128
    b = R.build(61, [n], [ql], H, 1, D, 16, dtype, fp8)
    b.update(k_scale=0.015 if fp8 else 1.0, v_scale=2.0 ** -6 if fp8 else 1.0)
    per = 8.0 * 128 * b["scale"] * b["k_scale"] / cap  # z of a key of ones
    b["q"] = torch.full_like(b["q"], 8.0)

    def stored(x):
        return torch.tensor(float(x)).to(torch.float8_e4m3fn if fp8 else b["dtype"]).view(torch.uint8 if fp8 else b["dtype"])

    b["kc"][:], b["vc"][:] = stored(0.0), stored(0.0)
    for j, at, v in ((10, z, 1.0), (74, z, -1.0), (80, -0.6, 0.0)):
        phys = b["tables"][0, j // 16]
        b["kc"][phys, :, j % 16] = stored(at / per)
        b["vc"][phys, :, j % 16] = stored(v / b["v_scale"])
    k = R.values(b, b["kc"], b["k_scale"])[b["tables"][0, 0], 0, 10, 0].item()
    assert 0.4 < 8.0 * 128 * b["scale"] * k / cap <= 0.5  # (as it is stored)
    return b


@pytest.mark.parametrize("cap", [20.0, 30.0, 50.0, 1000.0])
@pytest.mark.parametrize("dtype,fp8", [("bf16", True), ("f16", True), ("bf16", False), ("f16", False)])
def test_scores_near_half_the_cap(dtype, fp8, cap):
    check(capped_pair(cap, dtype, fp8, 0.48), softcap=cap)


@pytest.mark.parametrize("cap", [20.0, 30.0, 50.0])
@pytest.mark.parametrize("dtype,fp8", [("bf16", True), ("f16", True), ("bf16", False)])
def test_scores_near_half_the_cap_against_a_distance_bias(dtype, fp8, cap):
    """A far key near half the cap and the keys around each token, level with it by the distance bias."""
    b = capped_pair(cap, dtype, fp8, 0.48)
    top = cap * 0.446  # tanh(0.48)
    b["kc"][b["tables"][0, 4:6].long()] = 0  # (the second key and its neighbour)
    b["vc"][:] = 0xE8 if fp8 else -1.0  # (E4M3 codes of -64 and 64, times 2^-6)
    b["vc"][b["tables"][0, 0], :, 10] = 0x68 if fp8 else 1.0
    slopes = torch.tensor([(top - 2.3) / 225 * (1 + 0.02 * (h - 4)) for h in range(8)], dtype=torch.float32)
    check(b, softcap=cap, slopes=slopes)


@pytest.mark.parametrize("cap", [3e4, 2e5, 1e6, 1e12, 1e30])
@pytest.mark.parametrize("dtype,fp8", [("bf16", True), ("f16", True), ("bf16", False), ("f16", False)])
def test_caps_far_above_the_scale(dtype, fp8, cap):
    """Caps whose powers over the scale leave fp32's range, and half of which no score (of a 16-bit pool: one) reaches."""
    if cap < 1e5 and not fp8:
        check(capped_pair(cap, dtype, fp8, 0.48), softcap=cap)
    for qlens in (None, [40]):
        check(R.build(63, [256], qlens, 8, 1, 128, 16, dtype, fp8, spread=8.0), softcap=cap)


@pytest.mark.parametrize("scale", [1e-6, 1e3, -0.1, 0.0])
@pytest.mark.parametrize("dtype,fp8", [("bf16", True), ("f16", True), ("f16", False)])
def test_scales_far_from_the_cap(dtype, fp8, scale):
    """Scores far below and far beyond the cap, turned round, and all zero."""
    for qlens in (None, [40]):
        b = R.build(64, [200], qlens, 8, 1, 128, 16, dtype, fp8)
        b["scale"] = scale
        cap = 0.01 if scale == 1e-6 else 30.0
        # The tolerance's d_j = (D + 8) 2^-23 scale sum |q| |K| bounds an error's size only for scale >= 0 (below, it
        # is minus the bound). scale q.K = |scale| (-q).K, and -q is exact: the definition over the negated queries is
        # the same one, with d_j >= 0.
        ref, tol = R.reference(b if scale >= 0 else dict(b, q=-b["q"], scale=-scale), softcap=cap)
        assert R.worst(call(b, softcap=cap), ref, tol) <= 1.0


@pytest.mark.parametrize("dtype,fp8", [("bf16", True), ("f16", True), ("bf16", False)])
def test_the_largest_cap_is_no_cap(dtype, fp8):
    for qlens in (None, [40]):
        b = R.build(65, [200], qlens, 8, 1, 128, 16, dtype, fp8)
        ref, tol = R.reference(b)
        assert R.worst(call(b, softcap=1e30), ref, tol) <= 1.0


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", True), ("bf16", False)])
@pytest.mark.parametrize("qlens", [None, [20]])
def test_many_keys_below_the_smallest_16_bit_weight(dtype, fp8, qlens):
    """One key, and 16383 that weigh 2^-26 or 2^-24 of it each: below f16's steps, and together 2^-11 of the row."""
    n, H, D = 16384, 8, 128
    b = R.build(66, [n], qlens, H, 1, D, 16, dtype, fp8, spread=0.0)
    b["q"][:] = 0
    b["q"][:, :, 0] = 16.0
    b.update(scale=1.0, k_scale=0.0625 if fp8 else 1.0, v_scale=2.0 ** -6 if fp8 else 1.0)
    ln2 = 0.6931471805599453
    for name, low, top in (("kc", -25.0 * ln2 / 16, 0.0), ("vc", -1.0, 1.0)):
        per = b["k_scale"] if name == "kc" else b["v_scale"]
        kind = torch.float8_e4m3fn if fp8 else b["dtype"]
        pool = torch.zeros(b[name].shape, dtype=torch.float64)
        pool[..., 0] = low / per
        if name == "vc":
            pool[:] = low / per
        first = b["tables"][0, 0]
        pool[first, :, 3] = top / per
        b[name] = pool.to(kind).view(torch.uint8) if fp8 else pool.to(kind)
    check(b)


LONG = [  # H, Hkv, dtype, fp8, contexts, query lengths: contexts above 8192, split by the call itself or not at all
    (8, 2, "bf16", False, [16384, 9001], None), (8, 2, "f16", False, [16384, 9001], None),
    (8, 1, "bf16", True, [16384, 9001], None), (24, 1, "f16", False, [12000], None),
    (8, 1, "bf16", False, [16384, 70], [9, 40]), (8, 1, "f16", False, [16384, 70], [9, 40]),
    (8, 1, "bf16", True, [16384, 70], [9, 40]), (8, 1, "f16", True, [10000, 9000], [40, 3]),
]


@pytest.mark.parametrize("H,Hkv,dtype,fp8,ctx,qlens", LONG)
def test_long_contexts(H, Hkv, dtype, fp8, ctx, qlens):
    """Contexts of up to 16384 tokens, with the partitions that the call chooses."""
    b = R.build(67, ctx, qlens, H, Hkv, 128, 16, dtype, fp8)
    check(b, softcap=5.0)
    check(b, slopes=R.slopes_of(H) / 64, window=8200)


@pytest.mark.parametrize("B,dtype,fp8", [(8, "f16", False), (32, "bf16", True)])
def test_a_long_prompt(B, dtype, fp8):
    """700 tokens behind 8000 others under a document mask: many row tiles, each of many tiles of keys."""
    b = R.build(68, [8700], [700], 4, 1, 128, B, dtype, fp8)
    begin = [t * 11 % 8000 for t in range(700)]
    rows = list(range(0, 700, 23)) + [699]
    out = call(b, key_begin=begin, softcap=8.0)
    for t in rows:  # (row by row: the definition of a token alone)
        one = dict(b, ctx=[8000 + t + 1], qlens=[1], q=b["q"][t:t + 1], starts=[0, 1])
        ref, tol = R.reference(one, key_begin=[begin[t]], softcap=8.0)
        assert R.worst(out[t:t + 1], ref, tol) <= 1.0


def test_a_bad_value_that_all_rows_see_is_looked_for_once():
    """The same prompt by the medians of nine calls each: 0.21 ms clean, 1.19 ms with the NaN (one look over an item's
    values), and 59 ms where every row that came out non-finite is computed again: 20 times the clean call tells them
    apart."""
    n, H, Hkv, D, B = 4096, 16, 4, 128, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    kc, vc = (torch.randn((n // B, Hkv, B, D), device=DEV, dtype=torch.bfloat16, generator=g) for _ in range(2))
    q = torch.randn((n, H, D), device=DEV, dtype=torch.bfloat16, generator=g)
    tables = torch.arange(n // B, device=DEV, dtype=torch.int32)[None].contiguous()
    ctx, starts, out = i32([n]), i32([0, n]), torch.empty_like(q)
    medians = []
    for bad in (False, True):
        if bad:
            vc[0, :, 0] = float("nan")
        times = []
        for _ in range(9):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            binding.paged_attention_multi_query_scored(out, q, kc, vc, tables, ctx, starts, 0.1, softcap=9.0,
                                                       max_query_len=n, max_context_len=n)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        medians.append(sorted(times)[4])
    assert torch.isnan(out).all()
    assert medians[1] < 20 * medians[0]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [
    (32, 1, 128, 16, "f16", False), (33, 1, 128, 16, "bf16", False), (72, 2, 64, 8, "f16", False),
    (40, 1, 128, 16, "bf16", True), (41, 1, 128, 16, "bf16", True), (96, 2, 128, 32, "f16", True),
])
def test_decode_with_many_heads_on_a_kv_head(H, Hkv, D, B, dtype, fp8, rule):
    """On both sides of the rows from which the 256-row tile runs, and split over long contexts by the call."""
    b = R.build(69, [2600, 300, 0, 1, 77], None, H, Hkv, D, B, dtype, fp8)
    check(b, **rules_of(rule, b))


@pytest.mark.parametrize("H,q", [(4, 6), (4, 7), (8, 3), (8, 4), (8, 5), (8, 6)])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_workspace_serves_either_pool(H, q, fp8):
    """The size that the query gives is enough whichever tile the pool's type takes."""
    b = R.build(70, [2600, 1900], [q, q - 1], H, 1, 128, 16, "bf16", fp8)
    need = binding.paged_attention_scored_workspace_size(2 * q - 1, H, 1, 128, 16, q, 2600)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    ref, tol = R.reference(b, softcap=5.0)
    out = call(b, softcap=5.0, workspace=ws[:need] if need else None)
    assert R.worst(out, ref, tol) <= 1.0
    assert (ws[need:] == 0x5A).all() and binding.device_errors() == 0
