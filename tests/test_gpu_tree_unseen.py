"""Tree attention with blocks of drafted places that no token's mask names: their table entries may hold anything."""
import pytest
import torch

import scored_reference as R
import tree_reference as TR
from paged_kv_cache_91_gb300 import binding
from test_gpu_tree import call

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word(cuda_lib):
    binding.device_errors(clear=True)
    yield


@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [
    (2, 2, 128, 16, "bf16", False), (2, 2, 64, 8, "f16", False), (2, 2, 128, 16, "bf16", True),   # 8-column tile: 6 rows
    (8, 2, 128, 16, "bf16", False), (8, 2, 64, 8, "f16", False), (8, 2, 128, 32, "bf16", True)])  # 24 rows, and more
@pytest.mark.parametrize("committed", [[0, 60], [16, 33]])
def test_blocks_that_no_mask_names(committed, H, Hkv, D, B, dtype, fp8, part):
    """The blocks of drafted places alone, all but those that a mask names: none of them, the last one, one in between;
    the batch's second sequence has other masks than its first. A bad id that is seen is an error as before."""
    q = 6 if H == Hkv else 150
    b = TR.build(81, committed, [q, q], H, Hkv, D, B, dtype, fp8, W=5)
    tables = b["tables"].clone()
    for named in (set(), {q - 1}, {q // 2}):
        TR.set_mask(b, [set() if t % 3 == 0 else named for t in range(q)] + [set()] * q, W=5)
        b["tables"] = tables.clone()
        gone = []
        for s, c in enumerate(committed):
            for k in range(R.ceil_div(c, B), R.ceil_div(c + q, B)):
                if s == 1 or not any(k == (c + u) // B for u in named):
                    b["tables"][s, k] = [-1, b["kc"].shape[0], -(1 << 31), (1 << 31) - 1][k % 4]
                    gone.append((s, k))
        assert gone or len(named)
        ref, tol = TR.reference(b)
        assert R.worst(call(b, partition_size=part), ref, tol) <= 1.0
        assert binding.device_errors() == 0
    if gone:  # the last of them is named by one token
        s, k = gone[-1]
        u = max(0, k * B - committed[s])
        TR.set_mask(b, b["sets"][:q] + [{u} if t == q // 3 else set() for t in range(q)], W=5)
        ref, tol = TR.reference(b)
        assert R.worst(call(b, partition_size=part), ref, tol) <= 1.0
        assert binding.device_errors(clear=True) == 1
        begin = [0] * q + [committed[1] + u + 1] * q  # and hidden from it again
        ref, tol = TR.reference(b, key_begin=begin)
        assert R.worst(call(b, partition_size=part, key_begin=begin), ref, tol) <= 1.0
        assert binding.device_errors() == 0
