"""The workspace that a call makes for itself comes from its own stream's memory, whatever stream is current: memory
freed on the current stream may still be written by work queued there."""
import pytest
import torch

import scored_reference as R
from paged_kv_cache_91_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def calls(fp8):
    """name -> a call of stream, each of a kind that needs a workspace."""
    b = R.build(70, [900, 700], None, 8, 2, 128, 16, fp8=fp8)
    q, kc, vc, bt = (b[k].to(DEV) for k in ("q", "kc", "vc", "tables"))
    out, ctx, starts = torch.empty_like(q), i32(b["ctx"]), i32([0, 1, 2])
    f = "_fp8" if fp8 else ""
    scales = dict(k_scale=b["k_scale"], v_scale=b["v_scale"]) if fp8 else {}
    a, kw = (out, q, kc, vc), dict(scales, scale=b["scale"])
    part = dict(kw, max_context_len=900, partition_size=64)

    def of(name):
        return getattr(binding, name + f)

    return {
        "decode": lambda s: of("paged_attention_decode")(*a, bt, ctx, stream=s, **part),
        "multi_query": lambda s: of("paged_attention_multi_query")(*a, bt, ctx, starts, max_query_len=1, stream=s, **part),
        "shared_prefix": lambda s: of("paged_attention_decode_shared_prefix")(
            *a, bt[0, :2].contiguous(), 32, bt, i32([600, 600]), stream=s, **kw),
        "decode_scored": lambda s: of("paged_attention_decode_scored")(*a, bt, ctx, softcap=5.0, stream=s, **part),
        "multi_query_scored": lambda s: of("paged_attention_multi_query_scored")(
            *a, bt, ctx, starts, max_query_len=1, window=500, stream=s, **part),
    }


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", ["decode", "multi_query", "shared_prefix", "decode_scored", "multi_query_scored"])
def test_workspace_is_of_the_calls_stream(cuda_lib, monkeypatch, name, fp8):
    call = calls(fp8)[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def spy(*args, **kw):
        t = empty(*args, **kw)
        if t.dtype is torch.uint8 and t.is_cuda:
            made.append((torch.cuda.current_stream(), t.numel()))
        return t

    monkeypatch.setattr(torch, "empty", spy)
    for stream in (side, None, side):
        made.clear()
        call(stream)
        assert len(made) == 1 and made[0][1] > 0
        assert made[0][0] == (stream or torch.cuda.current_stream())
    torch.cuda.synchronize()


def test_memory_freed_on_the_current_stream_is_not_taken(cuda_lib, monkeypatch):
    """A block of the workspace's size, just freed on the current stream, stays with that stream."""
    call = calls(False)["decode_scored"]
    side, made, empty = torch.cuda.Stream(), [], torch.empty

    def spy(*args, **kw):
        made.append(empty(*args, **kw))
        return made[-1]

    monkeypatch.setattr(torch, "empty", spy)
    call(None)
    size = made[0].numel()
    made.clear()
    torch.cuda.synchronize()
    freed = empty(size, dtype=torch.uint8, device=DEV)
    at = freed.data_ptr()
    del freed
    call(side)
    assert made[0].numel() == size and made[0].data_ptr() != at
    torch.cuda.synchronize()


class Handle:
    """A stream of another library: a handle and no more."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("name", ["decode", "multi_query", "shared_prefix", "decode_scored", "multi_query_scored"])
def test_a_stream_known_by_its_handle(cuda_lib, name):
    call = calls(False)[name]
    want = call(None).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(Handle(side))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("wrap", [lambda s: s, Handle])
def test_the_longest_query_is_read_on_the_calls_stream(cuda_lib, scored, wrap):
    """query_start_loc is still being made on the call's stream when max_query_len is read from it."""
    b = R.build(71, [200, 90], [40, 1], 8, 2, 128, 16)
    ref, tol = R.reference(b)
    q, kc, vc, bt = (b[k].to(DEV) for k in ("q", "kc", "vc", "tables"))
    out, ctx, made = torch.full_like(q, float("nan")), i32(b["ctx"]), i32(b["starts"])
    starts = i32([0, 1, 2])
    fn = binding.paged_attention_multi_query_scored if scored else binding.paged_attention_multi_query
    side = torch.cuda.Stream()
    binding.device_errors(clear=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # some 50 ms
        starts.copy_(made)
    fn(out, q, kc, vc, bt, ctx, starts, b["scale"], max_context_len=200, stream=wrap(side))
    torch.cuda.synchronize()
    assert R.worst(out, ref, tol) <= 1.0
    assert binding.device_errors() == 0
