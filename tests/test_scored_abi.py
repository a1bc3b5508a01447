"""Scored attention and the block-table calls without a GPU: every refusal is made on the host."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_91_gb300 import binding
    from paged_kv_cache_91_gb300 import build as b

    b.build()
    return binding.load()


def fake(n):
    """A non-null, aligned address that is never dereferenced on the host path."""
    return P(0x10000 * n)


def decode(lib, fp8=False, **kw):
    a = dict(out=fake(1), query=fake(2), key_cache=fake(3), value_cache=fake(4), block_tables=fake(5),
             max_blocks_per_seq=8, context_lens=fake(6), num_seqs=2, max_context_len=128, scale=0.125, softcap=0.0,
             alibi_slopes=None, window=0, key_begin=None, block_size=16, num_heads=4, num_kv_heads=4, head_dim=128,
             num_blocks=16, dtype=0)
    if fp8:
        a.update(k_scale=0.5, v_scale=0.25)
    a.update(partition_size=0, workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    fn = lib.paged_attention_decode_scored_fp8 if fp8 else lib.paged_attention_decode_scored
    return fn(*a.values())


def multi_query(lib, fp8=False, **kw):
    a = dict(out=fake(1), query=fake(2), key_cache=fake(3), value_cache=fake(4), block_tables=fake(5),
             max_blocks_per_seq=8, context_lens=fake(6), query_start_loc=fake(7), num_seqs=2, num_query_tokens=5,
             max_query_len=4, max_context_len=128, scale=0.125, softcap=0.0, alibi_slopes=None, window=0,
             key_begin=None, key_end=None, block_size=16, num_heads=4, num_kv_heads=4, head_dim=128, num_blocks=16,
             dtype=0)
    if fp8:
        a.update(k_scale=0.5, v_scale=0.25)
    a.update(partition_size=0, workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    fn = lib.paged_attention_multi_query_scored_fp8 if fp8 else lib.paged_attention_multi_query_scored
    return fn(*a.values())


COMMON = [
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("nan")), INVALID), (dict(softcap=float("inf")), INVALID),
    (dict(softcap=1e-45, scale=1e30), INVALID),  # scale / softcap overflows
    (dict(window=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(num_heads=6), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(num_blocks=0), INVALID), (dict(max_blocks_per_seq=0), INVALID),
    (dict(max_context_len=-1), INVALID), (dict(max_context_len=129), INVALID), (dict(out=None), INVALID),
    (dict(context_lens=None), INVALID), (dict(query=P(0x20008)), INVALID), (dict(value_cache=P(0x40008)), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=70000), UNSUPPORTED), (dict(num_blocks=1 << 25), UNSUPPORTED),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", COMMON)
def test_decode_rejects_on_host(lib, kw, status, fp8):
    assert decode(lib, fp8, **kw) == status
    assert lib.pkv_last_error_message() != b""


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(query_start_loc=None), INVALID), (dict(num_query_tokens=-1), INVALID), (dict(max_query_len=-3), INVALID),
    (dict(max_query_len=129), INVALID), (dict(num_query_tokens=1 << 30), UNSUPPORTED),
])
def test_multi_query_rejects_on_host(lib, kw, status, fp8):
    assert multi_query(lib, fp8, **kw) == status
    assert lib.pkv_last_error_message() != b""


@pytest.mark.parametrize("call", [decode, multi_query])
@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=64), UNSUPPORTED), (dict(k_scale=0.0), INVALID), (dict(v_scale=-1.0), INVALID),
    (dict(k_scale=float("inf")), INVALID), (dict(v_scale=float("nan")), INVALID),
])
def test_fp8_rejects_on_host(lib, call, kw, status):
    assert call(lib, True, **kw) == status


def test_nothing_to_do_is_a_noop(lib):
    for fp8 in (False, True):
        assert decode(lib, fp8, num_seqs=0, out=None) == OK
        assert multi_query(lib, fp8, num_seqs=0, out=None) == OK
        assert multi_query(lib, fp8, num_query_tokens=0, out=None) == OK
        assert multi_query(lib, fp8, max_query_len=0, out=None) == OK


def reserve(lib, **kw):
    a = dict(block_tables=fake(1), max_blocks_per_seq=8, context_lens=fake(2), new_lens=fake(3), free_blocks=fake(4),
             free_capacity=4, num_free=fake(5), slot_mapping=fake(6), max_tokens=9, query_start_loc=fake(7),
             context_lens_out=fake(8), num_free_out=fake(9), granted=fake(10), num_seqs=3, block_size=16,
             num_blocks=8, stream=None)
    a.update(kw)
    return lib.paged_kv_reserve_slots(*a.values())


def release(lib, **kw):
    a = dict(block_tables=fake(1), max_blocks_per_seq=8, context_lens=fake(2), finished=fake(3), free_blocks=fake(4),
             free_capacity=4, num_free=fake(5), context_lens_out=fake(8), num_free_out=fake(9), num_seqs=3,
             block_size=16, num_blocks=8, stream=None)
    a.update(kw)
    return lib.paged_kv_release_blocks(*a.values())


SLOTS = [
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=70000), UNSUPPORTED), (dict(block_size=12), UNSUPPORTED),
    (dict(num_blocks=0), INVALID), (dict(max_blocks_per_seq=0), INVALID), (dict(free_capacity=-1), INVALID),
    (dict(max_blocks_per_seq=1 << 27), UNSUPPORTED), (dict(block_tables=None), INVALID),
    (dict(num_free=None), INVALID), (dict(num_free_out=None), INVALID), (dict(free_blocks=None), INVALID),
    (dict(context_lens_out=None), INVALID), (dict(context_lens_out=fake(2)), INVALID),
    (dict(context_lens_out=P(0x20008)), INVALID), (dict(num_free_out=fake(5)), INVALID),
]


@pytest.mark.parametrize("kw,status", SLOTS + [
    (dict(max_tokens=-1), INVALID), (dict(slot_mapping=None), INVALID), (dict(query_start_loc=None), INVALID),
    (dict(granted=None), INVALID), (dict(granted=fake(2)), INVALID), (dict(granted=P(0x30004)), INVALID),
    (dict(new_lens=None), INVALID),
])
def test_reserve_rejects_on_host(lib, kw, status):
    assert reserve(lib, **kw) == status
    assert lib.pkv_last_error_message() != b""


@pytest.mark.parametrize("kw,status", SLOTS + [(dict(finished=None), INVALID), (dict(context_lens_out=fake(3)), INVALID)])
def test_release_rejects_on_host(lib, kw, status):
    assert release(lib, **kw) == status
    assert lib.pkv_last_error_message() != b""


def test_binding_refuses_cpu_tensors(lib):
    from paged_kv_cache_91_gb300 import binding

    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    kc = torch.zeros(4, 4, 16, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    t = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(binding.PagedKVError):
        binding.paged_attention_decode_scored(x, x, kc, kc, t, i, 0.125, softcap=5.0)
    with pytest.raises(binding.PagedKVError):
        binding.paged_attention_multi_query_scored(x, x, kc, kc, t, i, torch.zeros(3, dtype=torch.int32), 0.125)
    with pytest.raises(binding.PagedKVError):
        binding.paged_kv_reserve_slots(t, i, i, i, one, torch.zeros(4, dtype=torch.int64),
                                       torch.zeros(3, dtype=torch.int32), i.clone(), one.clone(), i.clone(), 16, 4)
    with pytest.raises(binding.PagedKVError):
        binding.paged_kv_release_blocks(t, i, i, i, one, i.clone(), one.clone(), 16, 4)


def test_workspace_is_allocated_on_the_calls_stream(monkeypatch):
    """The workspace that a call makes is taken while the call's stream is the current one."""
    import contextlib

    from paged_kv_cache_91_gb300 import binding

    now = ["current"]

    @contextlib.contextmanager
    def stream_context(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    made, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (made.append(now[0]), empty(*a, **kw))[1])
    like = torch.zeros(1)
    assert binding._new_workspace(48, like, "side").shape == (48,)
    assert binding._new_workspace(32, like, None).dtype is torch.uint8
    assert made == ["side", "current"] and now == ["current"]


# Bytes of each array of a call of 3 sequences, tables of 8 entries, 4 free blocks and 9 tokens.
RESERVE_WRITES = dict(block_tables=96, slot_mapping=72, query_start_loc=16, context_lens_out=12, num_free_out=4, granted=12)
RESERVE_READS = dict(context_lens=12, new_lens=12, free_blocks=16, num_free=4)
RELEASE_WRITES = dict(free_blocks=16, context_lens_out=12, num_free_out=4)
RELEASE_READS = dict(block_tables=96, context_lens=12, finished=12, num_free=4)


@pytest.mark.parametrize("call,writes,reads", [(reserve, RESERVE_WRITES, RESERVE_READS),
                                               (release, RELEASE_WRITES, RELEASE_READS)])
def test_what_is_written_overlaps_nothing(lib, call, writes, reads):
    """An array that is written, laid over the last or the first bytes of any other one, is refused."""
    sizes = {**writes, **reads}
    for w in writes:
        for other, n in sizes.items():
            if other == w:
                continue
            at = 0x10000 * 99
            step = 8 if w == "slot_mapping" else 4  # one element
            for over in ((at + n - 1) // step * step, at - sizes[w] + step):
                assert call(lib, **{w: P(over), other: P(at)}) == INVALID, (w, other)
                message = lib.pkv_last_error_message().decode()
                assert "overlap" in message and w in message and other in message


def test_arrays_side_by_side_are_not_refused_as_overlapping(lib):
    """Neighbours in one allocation, with nothing between them, and empty arrays at another one's address, pass the
    check (a call without a place for its totals is refused for that alone)."""
    at, a = 0x20000, {}
    for name, n in {**RESERVE_WRITES, **RESERVE_READS}.items():
        if name == "slot_mapping":
            at = (at + 7) // 8 * 8
        a[name] = P(at)
        at += n
    assert reserve(lib, **a, block_size=12) == UNSUPPORTED
    none = dict(a, num_seqs=0, free_capacity=0, max_tokens=0, block_tables=None, slot_mapping=None, granted=a["num_free"],
                context_lens=a["num_free"], free_blocks=a["num_free_out"])
    for kw in (a, none):
        reserve(lib, **kw)  # (refused for want of a device here, if at all)
        assert b"overlap" not in lib.pkv_last_error_message()


@pytest.mark.parametrize("call", [decode, multi_query])
@pytest.mark.parametrize("fp8", [False, True])
def test_caps_whose_factors_leave_the_range_are_refused(lib, call, fp8):
    """2 log2(e) softcap has to be finite in fp32 (2.88 * 1.18e38 is not), and scale / softcap far from subnormal."""
    for cap in (1.1e30, 1e38, 3.4e38):
        assert call(lib, fp8, softcap=cap) == INVALID
        assert b"softcap" in lib.pkv_last_error_message()
    assert call(lib, fp8, softcap=1e30, num_seqs=0) == OK


@pytest.mark.parametrize("fp8", [False, True])
def test_a_grid_of_empty_places_is_refused(lib, fp8):
    """max_query_len times the sequences: 2^27 places for row tiles, and no more (2048 of them a sequence and kv head)."""
    kw = dict(num_heads=32, num_kv_heads=8, max_query_len=131072, max_context_len=131072, max_blocks_per_seq=8192,
              num_query_tokens=65535)
    assert multi_query(lib, fp8, **kw, num_seqs=8193) == UNSUPPORTED
    assert b"max_query_len" in lib.pkv_last_error_message()
    assert multi_query(lib, fp8, **kw, num_seqs=8192, out=None) == INVALID  # (the next check)
    assert multi_query(lib, fp8, **dict(kw, max_query_len=4), num_seqs=65535, out=None) == INVALID
    assert multi_query(lib, fp8, **dict(kw, max_query_len=524280, max_context_len=1 << 30, max_blocks_per_seq=1 << 27,
                                        num_query_tokens=1 << 20), num_seqs=65535) == UNSUPPORTED


def test_release_refuses_more_blocks_than_it_counts(lib):
    """A CTA counts its sequences' blocks in 32 bits: tables of 2^31 entries for the sequences of one are refused."""
    apart = ("context_lens", "finished", "free_blocks", "num_free", "context_lens_out", "num_free_out")
    kw = dict({n: P((i + 1) << 24) for i, n in enumerate(apart)}, block_size=8, block_tables=P(1 << 44))
    wide = (1 << 28) - 16
    assert release(lib, num_seqs=304 * 8 + 1, max_blocks_per_seq=wide, **kw) == UNSUPPORTED
    assert b"2^31" in lib.pkv_last_error_message()
    assert release(lib, num_seqs=65535, max_blocks_per_seq=(1 << 31) // 216 + 1, **kw) == UNSUPPORTED
    release(lib, num_seqs=304 * 7, max_blocks_per_seq=wide, **kw)  # (seven sequences: not for that)
    assert b"2^31" not in lib.pkv_last_error_message()
