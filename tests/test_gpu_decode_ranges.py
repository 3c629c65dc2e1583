"""The decode step's operators at the ends of their types' ranges: values, scales and caps far from
ordinary sizes, NaN markers, and the layouts that only long rows reach.  Against the float64 oracle.

Attention's bounds are those of test_gpu_kv_cache.py, with tighter ones for lse: weights are summed in float32,
unrounded, so that lse is off by what the scores are off by (dz), the sum's roundings (a lane adds less than 2^7
weights one after the other here: 2^-17) and its own last places.
"""
import numpy as np
import pytest
import torch

from oracle import bf16, decode
from w4a16_group_quantized_w4_b200 import api
from tests._util import dev_bf16, host_bf16_bits, host_f64
from tests.test_gpu_kv_cache import KINDS, host_codes, stored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_rows_of_every_size_are_read_back_whole(kind):
    """s * q of every finite group, rounded once; scales from the smallest subnormal to 2^120 (int8), 2^125 (int4)."""
    r = np.random.RandomState(12)
    T, dim = 600, 64
    size = np.concatenate([r.randint(-133, 128, T - 40), np.full(40, 126)])
    k, v = (bf16.from_f64(np.clip(r.randn(T, 1, dim) * 2.0 ** size[:, None, None], -3e38, 3e38)) for _ in range(2))
    k[5, 0, 32:] = 0                                   # zeros beside a large group, and codes 0 inside one
    k[-1, 0, 1:32] = 0
    cache = api.KVCache(T, 1, 1, dim, kind)
    slots = torch.arange(T, device="cuda")
    cache.write(dev_bf16(k), dev_bf16(v), slots)
    for x, got in zip((k, v), cache.read(slots)):
        q, s = decode.quantise_rows(x.reshape(-1, dim), kind)
        assert bf16.to_f64(s).max() > 2.0 ** 118
        assert np.array_equal(host_bf16_bits(got).reshape(T, dim), bf16.from_f64(decode.row_values(q, s)))
