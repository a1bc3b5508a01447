"""The calls of a speculative step on trees without a GPU: every refusal is made on the host."""
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
    return P(0x1000000 * n)


def tree(lib, fp8=False, **kw):
    a = dict(out=fake(1), query=fake(2), key_cache=fake(3), value_cache=fake(4), block_tables=fake(5),
             max_blocks_per_seq=8, context_lens=fake(6), query_start_loc=fake(7), num_seqs=2, num_query_tokens=5,
             max_query_len=4, max_context_len=128, tree_mask=fake(8), mask_words=1, scale=0.125, softcap=0.0,
             key_begin=None, block_size=16, num_heads=4, num_kv_heads=4, head_dim=128, num_blocks=16, dtype=0)
    if fp8:
        a.update(k_scale=0.5, v_scale=0.25)
    a.update(partition_size=0, workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    return (lib.paged_attention_tree_fp8 if fp8 else lib.paged_attention_tree)(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("nan")), INVALID), (dict(softcap=2e30), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(num_heads=6), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(num_blocks=0), INVALID), (dict(max_blocks_per_seq=0), INVALID), (dict(max_context_len=-1), INVALID),
    (dict(max_context_len=129), INVALID), (dict(out=None), INVALID), (dict(context_lens=None), INVALID),
    (dict(tree_mask=None), INVALID), (dict(mask_words=0), INVALID), (dict(mask_words=-1), INVALID),
    (dict(max_query_len=33), INVALID), (dict(max_query_len=129, mask_words=5), INVALID), (dict(query=P(0x2000008)), INVALID),
    (dict(query_start_loc=None), INVALID), (dict(num_query_tokens=-1), INVALID), (dict(max_query_len=-3), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=70000), UNSUPPORTED), (dict(num_blocks=1 << 25), UNSUPPORTED),
    (dict(num_query_tokens=1 << 30), UNSUPPORTED), (dict(partition_size=24), UNSUPPORTED),
    (dict(partition_size=16), WORKSPACE),
])
def test_tree_rejects_on_host(lib, kw, status, fp8):
    assert tree(lib, fp8, **kw) == status
    assert lib.pkv_last_error_message() != b""


def test_tree_fp8_rejects_on_host(lib):
    for kw, status in ((dict(head_dim=64), UNSUPPORTED), (dict(k_scale=0.0), INVALID), (dict(v_scale=float("nan")), INVALID)):
        assert tree(lib, True, **kw) == status


def test_tree_of_nothing_is_a_noop(lib):
    for fp8 in (False, True):
        for kw in (dict(num_seqs=0), dict(num_query_tokens=0), dict(max_query_len=0, mask_words=0)):
            assert tree(lib, fp8, out=None, **kw) == OK


def rope(lib, fp8=False, **kw):
    a = dict(query_out=fake(1), query=fake(2), key=fake(3), value=fake(4), key_cache=fake(5), value_cache=fake(6),
             slot_mapping=fake(7), positions=fake(8), cos_sin=fake(9), max_position=100, rotary_dim=128, interleaved=0,
             q_weight=fake(10), k_weight=None, eps=1e-6, num_tokens=3, query_stride=1024, key_stride=1024,
             value_stride=1024, num_heads=4, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=8, dtype=1)
    if fp8:
        a.update(k_scale=0.5, v_scale=0.25)
    a.update(stream=None)
    a.update(kw)
    return (lib.paged_kv_write_rope_fp8 if fp8 else lib.paged_kv_write_rope)(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(num_tokens=-1), INVALID), (dict(dtype=2), INVALID), (dict(num_heads=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_blocks=0), INVALID), (dict(num_heads=65536, query_stride=1 << 23), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(block_size=64), UNSUPPORTED), (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=144), INVALID),
    (dict(rotary_dim=24), UNSUPPORTED), (dict(max_position=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(query_stride=504), INVALID), (dict(query_stride=1025), INVALID),
    (dict(key_stride=128), INVALID), (dict(value_stride=1028), INVALID), (dict(key_stride=(1 << 31) + 8), UNSUPPORTED),
    (dict(query_out=None), INVALID), (dict(slot_mapping=None), INVALID), (dict(positions=None), INVALID),
    (dict(cos_sin=None), INVALID), (dict(cos_sin=P(0x9000004)), INVALID), (dict(q_weight=P(0xa000004)), INVALID),
    (dict(k_weight=P(0xa000008)), INVALID), (dict(key=P(0x3000008)), INVALID),
    (dict(query_out=P(0x2000000)), INVALID),        # query itself, but with gaps
    (dict(query_out=P(0x2000100)), INVALID), (dict(query_out=P(0x2000100), query_stride=512), INVALID),
    (dict(query_out=P(0x3000800)), INVALID), (dict(query_out=P(0x3fffff0)), INVALID),
])
def test_rope_rejects_on_host(lib, kw, status, fp8):
    assert rope(lib, fp8, **kw) == status
    assert lib.pkv_last_error_message() != b""


def test_rope_fp8_rejects_scales(lib):
    for kw in (dict(k_scale=0.0), dict(k_scale=float("inf")), dict(v_scale=-1.0), dict(v_scale=float("nan"))):
        assert rope(lib, True, **kw) == INVALID


def test_rope_of_nothing_is_a_noop(lib):
    assert rope(lib, num_tokens=0, query_out=None) == OK


def layout(lib, **kw):
    a = dict(parents=fake(1), query_start_loc=fake(2), context_lens=fake(3), num_seqs=2, num_query_tokens=9,
             max_query_len=5, tree_mask=fake(4), mask_words=1, positions=fake(5), stream=None)
    a.update(kw)
    return lib.paged_kv_tree_layout(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), INVALID), (dict(num_query_tokens=-1), INVALID), (dict(max_query_len=-1), INVALID),
    (dict(mask_words=-1), INVALID), (dict(max_query_len=33), INVALID), (dict(max_query_len=1025, mask_words=33), UNSUPPORTED),
    (dict(num_seqs=65536), UNSUPPORTED), (dict(parents=None), INVALID), (dict(positions=None), INVALID),
    (dict(tree_mask=None), INVALID), (dict(positions=P(0x1000010)), INVALID), (dict(positions=P(0x4000020)), INVALID),
    (dict(tree_mask=P(0x2000008)), INVALID), (dict(tree_mask=P(0x2ffffe0)), INVALID),
])
def test_layout_rejects_on_host(lib, kw, status):
    assert layout(lib, **kw) == status
    assert lib.pkv_last_error_message() != b""


def test_layout_of_nothing_is_a_noop(lib):
    for kw in (dict(num_seqs=0), dict(num_query_tokens=0), dict(max_query_len=0)):
        assert layout(lib, parents=None, **kw) == OK


def compact(lib, **kw):
    a = dict(key_cache=fake(1), value_cache=fake(2), num_layers=3, block_tables=fake(3), max_blocks_per_seq=8,
             context_lens=fake(4), query_start_loc=fake(5), num_seqs=2, accepted=fake(6), max_accepted=4,
             num_accepted=fake(7), num_kv_heads=2, head_dim=128, block_size=16, num_blocks=8, dtype=2, stream=None)
    a.update(kw)
    return lib.paged_kv_compact_accepted(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(num_layers=-1), INVALID), (dict(num_seqs=-1), INVALID), (dict(max_accepted=-1), INVALID), (dict(dtype=3), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(num_blocks=0), INVALID), (dict(max_blocks_per_seq=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED), (dict(num_seqs=65536), UNSUPPORTED),
    (dict(num_blocks=1 << 27), UNSUPPORTED), (dict(num_layers=1 << 30), UNSUPPORTED), (dict(key_cache=None), INVALID),
    (dict(num_accepted=None), INVALID), (dict(value_cache=P(0x2000008)), INVALID),
])
def test_compact_rejects_on_host(lib, kw, status):
    assert compact(lib, **kw) == status
    assert lib.pkv_last_error_message() != b""


def test_compact_of_nothing_is_a_noop(lib):
    for kw in (dict(num_layers=0), dict(num_seqs=0), dict(max_accepted=0)):
        assert compact(lib, key_cache=None, **kw) == OK


def trim(lib, **kw):
    a = dict(block_tables=fake(1), max_blocks_per_seq=8, context_lens=fake(2), keep_lens=fake(3), free_blocks=fake(4),
             free_capacity=4, num_free=fake(5), context_lens_out=fake(8), num_free_out=fake(9), num_seqs=3,
             block_size=16, num_blocks=8, stream=None)
    a.update(kw)
    return lib.paged_kv_trim_blocks(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), INVALID), (dict(num_blocks=0), INVALID), (dict(max_blocks_per_seq=0), INVALID),
    (dict(free_capacity=-1), INVALID), (dict(block_size=64), UNSUPPORTED), (dict(num_seqs=65536), UNSUPPORTED),
    (dict(keep_lens=None), INVALID), (dict(num_free=None), INVALID), (dict(context_lens_out=fake(3)), INVALID),
    (dict(num_free_out=fake(5)), INVALID), (dict(free_blocks=fake(1)), INVALID), (dict(context_lens_out=fake(2)), INVALID),
])
def test_trim_rejects_on_host(lib, kw, status):
    assert trim(lib, **kw) == status
    assert lib.pkv_last_error_message() != b""


def test_workspace_size(lib):
    size = lib.paged_attention_tree_workspace_size
    assert size(40, 8, 2, 128, 16, 20, 4096, 1024) == 40 * 8 * 4 * 130 * 4
    assert size(40, 8, 2, 128, 16, 20, 1024, 1024) == 0
    for bad in ((0, 8, 2, 128, 16, 20, 4096, 0), (40, 8, 3, 128, 16, 20, 4096, 0), (40, 8, 2, 128, 16, 0, 4096, 0)):
        assert size(*bad) == 0


def test_binding_wants_cuda_tensors():
    from paged_kv_cache_91_gb300 import binding

    x, i = torch.zeros(1, 1, 64, dtype=torch.float16), torch.zeros(1, dtype=torch.int32)
    pool, slots = torch.zeros(1, 1, 16, 64, dtype=torch.float16), torch.zeros(1, dtype=torch.int64)
    two = torch.zeros(2, dtype=torch.int32)
    for call in (
        lambda: binding.paged_kv_write_rope(x, x, x, x, pool, pool, slots, None, None),
        lambda: binding.paged_attention_tree(x, x, pool, pool, i[None], i, two, i[None], 1.0),
        lambda: binding.paged_kv_tree_layout(i, two, i, i[None], i),
        lambda: binding.paged_kv_compact_accepted(pool, pool, i[None], i, two, i[None], i),
        lambda: binding.paged_kv_trim_blocks(i[None], i, i, i, i, i, i, 16, 1),
    ):
        with pytest.raises(binding.PagedKVError):
            call()
