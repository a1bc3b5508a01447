"""Tree attention whose CTAs take many small items one after the other."""
import random

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


@pytest.mark.parametrize("H,Hkv,D,B,dtype,fp8", [(40, 4, 128, 16, "bf16", False), (72, 8, 64, 8, "f16", False),
                                                 (40, 4, 128, 32, "bf16", True), (36, 4, 128, 16, "f16", True)])
def test_items_of_one_tile(H, Hkv, D, B, dtype, fp8):
    """Some ten items a CTA, most of them of one tile of 64 keys, in which the second stream has no part, with one of
    several tiles now and then."""
    r = random.Random(61)
    committed = [r.choice([0, 3, 30, 50]) if r.random() < 0.9 else r.randint(64, 300) for _ in range(400)]
    b = TR.build(61, committed, [1] * len(committed), H, Hkv, D, B, dtype, fp8)
    ref, tol = TR.reference(b)
    want = call(b)
    assert R.worst(want, ref, tol) <= 1.0
    for _ in range(20):
        assert torch.equal(call(b), want)
    assert binding.device_errors() == 0
