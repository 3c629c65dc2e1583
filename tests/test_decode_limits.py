"""Limits of the decode step's operators that the host checks (CPU only: before any CUDA call)."""
import pytest
import torch

from w4a16_group_quantized_w4_b200 import _lib, api, stack

P = 4096            # a well aligned, never dereferenced address


@pytest.mark.parametrize("M,K", [(33, 32), (40, 64), (17, 4928), (32, 8192), (16, 11040), (1, 23072), (600, 8192)])
def test_linear8_weight_rows_of_the_tiled_kernel(M, K):
    """Calls that neither the kernel of few rows nor the tensor-memory kernel takes: up to 65535 tiles of 128."""
    lib = _lib.load()
    assert lib.w4a8_linear(P, P, P, P, P, M, 65535 * 128 + 1, K, P, 1 << 60, None) == _lib.W4_ERR_UNSUPPORTED


@pytest.mark.parametrize("dim", [32, 96, 160, 512])
@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_block_refuses_a_cache_that_attention_does_not_take(dim, kind):
    """At once, not at its first step."""
    cache = api.KVCache(2, 1, 16, dim, kind, device="cpu")
    w = [torch.zeros((4 * dim, 8), dtype=torch.int32), torch.zeros((4 * dim, 2), dtype=torch.bfloat16),
         torch.zeros((64, 2 * dim // 8), dtype=torch.int32), torch.zeros((64, 2 * dim // 32), dtype=torch.bfloat16)]
    with pytest.raises(ValueError, match="head_dim"):
        stack.AttentionBlock(*w, cache, 2)


def test_block_takes_the_others():
    for dim in (64, 128, 192, 256):
        w = [torch.zeros((4 * dim, 8), dtype=torch.int32), None, torch.zeros((64, 2 * dim // 8), dtype=torch.int32), None]
        assert stack.AttentionBlock(*w, api.KVCache(2, 1, 16, dim, "int8", device="cpu"), 2).dim == dim
