"""Device-side failure detection of w4a8_linear, exercised without a GPU fault.

Every wait of its kernels on an mbarrier is bounded; when the limit runs out they report W4_ERR_TIMEOUT, ask for no
further copies, wait for the ones on their way and return, with NaN in what the lost data would have fed.  The
library's fault-injection export (not part of w4a16.h) leaves out every ring's copies from a given stage on, with a
20 ms limit (2 s, as always, in the tensor-memory kernel).
"""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import decode
from w4a16_group_quantized_w4_b200 import _lib, api
from tests._util import dev_bf16, dev_u32, host_f64
from tests.test_gpu_rms_add import linear_case

pytestmark = pytest.mark.gpu


def stalled(xq, xs, codes, scales, stall_after, wait_ns=20_000_000):
    """-> (y, status) of a call that loses every stage from stall_after on."""
    fn = _lib.load().w4_testing_linear8_stall
    P, I64 = C.c_void_p, C.c_int64
    fn.restype = C.c_int32
    fn.argtypes = [P, P, P, P, P, I64, I64, I64, P, C.c_size_t, P, P, C.c_uint64, C.c_int32]
    M, K = xq.shape
    N = codes.shape[0]
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    need = api.w4_workspace_bytes(_lib.W4_OP_LINEAR_8, M, N, K, 1, 1)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert fn(xq.data_ptr(), xs.data_ptr(), codes.data_ptr(), scales.data_ptr(), y.data_ptr(), M, N, K, ws.data_ptr(), need,
              status.data_ptr(), torch.cuda.current_stream().cuda_stream, wait_ns, stall_after) == _lib.W4_OK
    torch.cuda.synchronize()
    return host_f64(y), status.item()


# up to 32 rows; tiles of 16, 32 and 64 tokens, with K split or not, scales by TMA or not
SHAPES = [(4, 14336, 4096), (30, 16384, 2080), (12, 64, 32768), (20, 300, 8192), (33, 72, 1024), (65, 300, 1120)]
# the tensor-memory kernel: token blocks of 192 and of 256, blocks of one tile and of several
MANY = [(900, 5632, 1024), (300, 16384, 832), (509, 8192, 2816), (257, 9472, 2048)]


@pytest.mark.parametrize("M,N,K,stall_after", [(*s, n) for s in SHAPES for n in (0, 1, 3)] +
                         [(*s, n) for s, n in zip(MANY, (9, 3, 20, 0))])
def test_lost_copies_are_reported_and_leave_nan(M, N, K, stall_after):
    xq, xs, codes, scales = linear_case(M, N, K, M)
    a = torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), dev_u32(codes), dev_bf16(scales)
    want = host_f64(api.w4a8_linear(*a))
    got, status = stalled(*a, stall_after)
    lost = np.isnan(got)
    assert np.array_equal(got[~lost], want[~lost])
    assert status == (_lib.W4_ERR_TIMEOUT if lost.any() else _lib.W4_OK)
    assert lost.all() if stall_after == 0 else True
    # the context is usable and the next call's results are right
    assert np.array_equal(host_f64(api.w4a8_linear(*a)), want)


@pytest.mark.parametrize("M,N,K", SHAPES + MANY)
def test_nothing_is_reported_when_nothing_is_lost(M, N, K):
    xq, xs, codes, scales = linear_case(M, N, K, M)
    a = torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), dev_u32(codes), dev_bf16(scales)
    got, status = stalled(*a, 1 << 30, 2_000_000_000)
    assert status == _lib.W4_OK and np.array_equal(got, host_f64(api.w4a8_linear(*a)))
    if (M, N, K) in MANY:                       # (the oracle's part: test_linear_many_rows)
        return
    ref, mag = decode.w4a8_linear(xq, xs, codes, scales), decode.w4a8_magnitude(xq, xs, codes, scales)
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (K // 32 + 4) * 2.0 ** -24 * 1.01).all()


@pytest.mark.parametrize("M,N,K", [SHAPES[0], SHAPES[3], MANY[0]])
def test_status_word_of_the_call(M, N, K):
    xq, xs, codes, scales = linear_case(M, N, K, M)
    a = torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), dev_u32(codes), dev_bf16(scales)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(api.w4a8_linear(*a, dev_status=status), api.w4a8_linear(*a)) and status.item() == 0
    with pytest.raises(TypeError):
        api.w4a8_linear(*a, dev_status=status.long())
    with pytest.raises(ValueError):
        api.w4a8_linear(*a, dev_status=torch.zeros(2, dtype=torch.int32, device="cuda"))
