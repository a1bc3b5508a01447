"""paged_kv_write_rope over its own queries, where a thread's later rows load behind the stores of its earlier ones."""
import pytest
import torch

from paged_kv_cache_91_gb300 import binding
from test_gpu_rope import call, make, near16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word(cuda_lib):
    binding.device_errors(clear=True)
    yield


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("H,Hkv,D,B", [(100, 4, 128, 16), (71, 71, 128, 8), (150, 2, 64, 32)])
def test_many_heads_in_place(H, Hkv, D, B, dtype, fp8, interleaved):
    c = make(91, 700, H, Hkv, D, B, dtype, fp8)
    want, kc, vc = call(c, interleaved)
    near16(c, want, c["q"], c["qw"], interleaved)
    out, kc2, vc2 = call(c, interleaved, out=c["q"])
    assert torch.equal(out, want) and torch.equal(kc.view(torch.uint8), kc2.view(torch.uint8))
    assert torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
    assert binding.device_errors() == 0
