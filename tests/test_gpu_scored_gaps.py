"""Scored attention whose tokens' intervals leave blocks between them that none sees: their table entries may hold
anything."""
import pytest
import torch

import scored_reference as R
from paged_kv_cache_91_gb300 import binding
from test_gpu_scored import call

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word(cuda_lib):
    binding.device_errors(clear=True)
    yield


@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [
    (2, 2, 128, 16, "bf16", False), (2, 2, 64, 8, "f16", False), (2, 2, 128, 16, "bf16", True),  # 8-column tile: 6 rows
    (16, 2, 128, 16, "bf16", False), (16, 2, 64, 8, "f16", False), (16, 2, 128, 32, "bf16", True)])  # 48 rows
def test_blocks_between_intervals(H, Hkv, D, B, dtype, fp8):
    q, n = 6, 400
    b = R.build(82, [n, n], [q, q], H, Hkv, D, B, dtype, fp8)
    begin, end = [0, 3, 300, 301, 350, 0] * 2, [40, 30, 350, 310, 400, 10] * 2
    for s in range(2):
        b["tables"][s, R.ceil_div(40, B):300 // B] = [-1, b["kc"].shape[0]][s]
    ref, tol = R.reference(b, key_begin=begin, key_end=end)
    assert R.worst(call(b, key_begin=begin, key_end=end), ref, tol) <= 1.0
    assert binding.device_errors() == 0
    end[1] = 10 * B + 1  # a block of them is seen
    ref, tol = R.reference(b, key_begin=begin, key_end=end)
    assert R.worst(call(b, key_begin=begin, key_end=end), ref, tol) <= 1.0
    assert binding.device_errors() == 1
