"""Limits of the decode step's operators that the host checks (CPU only: before any CUDA call)."""
import pytest

from w4a16_group_quantized_w4_b200 import _lib

P = 4096            # a well aligned, never dereferenced address


@pytest.mark.parametrize("M,K", [(33, 32), (40, 64), (17, 4928), (32, 8192), (16, 11040), (1, 23072), (600, 8192)])
def test_linear8_weight_rows_of_the_tiled_kernel(M, K):
    """Calls that neither the kernel of few rows nor the tensor-memory kernel takes: up to 65535 tiles of 128."""
    lib = _lib.load()
    assert lib.w4a8_linear(P, P, P, P, P, M, 65535 * 128 + 1, K, P, 1 << 60, None) == _lib.W4_ERR_UNSUPPORTED
