"""GPU parity of w4_rms_add, w4_rms_add_q8 and w4a8_linear against the float64 oracle.

Tolerances (derived, per element):
  * bf16 outputs are rounded once: half a step is 2^-8 of the value at most.
  * the float32 chain in front of it (sum of squares in any order, division, root, two products) is
    within (H / 8 + 16) * 2^-24 relative: partial sums of at most H/8 terms a thread plus the tree.
  * 8-bit rows: |y / s - q| <= 1/2 plus the chain's error times 127.
  * w4a8: group sums are exact, the accumulation of G groups is within (G + 4) * 2^-24 of the sum of
    the groups' magnitudes, then one bf16 rounding.  Many rows go to the tensor-memory kernel, which sums
    16 exact products a step in float32: within (K / 16) * 2^-23 of the sum of all magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import bf16, decode
from w4a16_group_quantized_w4_b200 import _lib, api
from tests._util import dev_bf16, dev_u32, host_bf16_bits, host_f64

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8


def chain(H):
    return (H / 8 + 16) * 2.0 ** -24


def case(T, H, seed, residual=True, weight=True, size=1.0):
    r = np.random.RandomState(seed)
    x = bf16.from_f64(size * r.randn(T, H))
    res = bf16.from_f64(3 * size * r.randn(T, H)) if residual else None
    w = bf16.from_f64(1 + 0.3 * r.randn(H)) if weight else None
    return x, res, w


def dev(a):
    return None if a is None else dev_bf16(a)


SIZES = [(1, 8), (1, 2816), (5, 64), (64, 2816), (3, 8 * 37), (301, 256), (700, 2816), (2, 8200), (400, 8200),
         (3, 16392), (2, 32768), (129, 1024)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False), (False, False)])
def test_bf16_rows(T, H, residual, weight):
    x, res, w = case(T, H, T + H, residual, weight)
    y, h = api.w4_rms_add(dev(x), dev(res), dev(w))
    h_ref, y_ref = decode.rms_add(x, res, w, api.RMS_EPS)
    assert np.array_equal(host_bf16_bits(h), h_ref)
    err = np.abs(host_f64(y) - y_ref)
    assert (err <= np.abs(y_ref) * (HALF_BF16 + 1.01 * chain(H))).all()


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("residual,weight", [(True, True), (False, False)])
def test_8bit_rows(T, H, residual, weight):
    x, res, w = case(T, H, T + H + 1, residual, weight)
    q, qs, h = api.w4_rms_add_q8(dev(x), dev(res), dev(w))
    h_ref, y_ref = decode.rms_add(x, res, w, api.RMS_EPS)
    assert np.array_equal(host_bf16_bits(h), h_ref)
    s_ref = np.abs(y_ref).max(axis=1) / 127
    s = qs.cpu().numpy().astype(np.float64)
    assert (np.abs(s - s_ref) <= s_ref * chain(H) * 1.01).all()
    qq = q.cpu().numpy().astype(np.float64)
    assert np.abs(qq).max() == 127
    assert (np.abs(qq - y_ref / s_ref[:, None]) <= 0.5 + 127 * 3 * chain(H)).all()


def test_rows_of_zeros_infinities_and_nan():
    x, res, w = case(6, 512, 5)
    x[1], res[1] = 0, 0
    x[2, 17] = 0x7F80
    x[3, 500] = 0x7FC0
    x[4], res[4] = bf16.from_f64(np.full(512, 1e-30)), 0
    q, qs, _ = api.w4_rms_add_q8(dev(x), dev(res), dev(w))
    y, _ = api.w4_rms_add(dev(x), dev(res), dev(w))
    q, qs, y = q.cpu().numpy(), qs.cpu().numpy(), host_f64(y)
    assert qs[1] == 0 and not q[1].any() and not y[1].any()
    for r in (2, 3):
        assert np.isnan(qs[r]) and not q[r].any()
    assert np.isnan(y[3]).all() and np.isnan(y[2, 17])
    good = [0, 4, 5]
    _, y_ref = decode.rms_add(x[good], res[good], w, api.RMS_EPS)
    assert (np.abs(y[good] - y_ref) <= np.abs(y_ref) * (HALF_BF16 + 1.01 * chain(512))).all()
    assert np.isfinite(qs[good]).all()


@pytest.mark.parametrize("wsize,xsize", [(1e-35, 1e-3), (5e-36, 1e-4), (1e-34, 1e-3), (1e30, 1e-3)])
def test_weights_at_the_ends_of_the_range(wsize, xsize):
    """Products h w so small that 127 / max|h w| is no float32 number, or subnormal themselves, under a scale
    that is a normal one; and large ones.  A subnormal product is off by 2^-150, which is 2^-21 of a largest
    one of at least 2^-129."""
    x, res, w = case(5, 512, 3)
    x, res = (bf16.from_f64(xsize * bf16.to_f64(t)) for t in (x, res))
    w = bf16.from_f64(wsize * bf16.to_f64(w))
    q, qs, h = api.w4_rms_add_q8(dev(x), dev(res), dev(w))
    _, y_ref = decode.rms_add(x, res, w, api.RMS_EPS)
    s_ref = np.abs(y_ref).max(axis=1) / 127
    assert (s_ref > 2.0 ** -126).all() and (np.abs(host_f64(h) * bf16.to_f64(w)).max(axis=1) > 2.0 ** -129).all()
    s = qs.cpu().numpy().astype(np.float64)
    slack = chain(512) + 2.0 ** -21
    assert (np.abs(s - s_ref) <= s_ref * slack * 1.01).all()
    qq = q.cpu().numpy().astype(np.float64)
    assert (np.abs(qq - y_ref / s_ref[:, None]) <= 0.5 + 127 * 3 * slack).all()


def test_residual_updated_in_place_and_rows_beside_left_alone():
    x, res, w = case(33, 2816, 9)
    want_y, want_h = api.w4_rms_add(dev(x), dev(res), dev(w))
    buf = torch.full((35, 2816), 7.0, dtype=torch.bfloat16, device="cuda")
    buf[1:34] = dev(res)
    h = buf[1:34]
    y, got_h = api.w4_rms_add(dev(x), h, dev(w), h=h)
    assert got_h is h and torch.equal(h, want_h) and torch.equal(y, want_y)
    assert (buf[0] == 7).all() and (buf[34] == 7).all()


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y, _ = api.w4_rms_add(x)
    q, qs, _ = api.w4_rms_add_q8(x)
    assert y.shape == (0, 64) and q.shape == (0, 64) and qs.shape == (0,)


def linear_case(M, N, K, seed, peak=False):
    r = np.random.RandomState(seed)
    xq = r.randint(-128, 128, (M, K)).astype(np.int8)
    q = r.randint(-8, 8, (N, K))
    if peak:                                      # the largest sums a group can have
        xq[:], q[:] = -128, -8
    s = bf16.from_f64((0.01 * np.abs(r.randn(N, K // 32)) + 1e-4) * np.exp(2 * r.randn(N, 1)))
    xs = (np.exp(r.randn(M)) / 127).astype(np.float32)
    return xq, xs, decode.pack_l1(q), s


def check_linear(xq, xs, codes, scales, scale_offset=0):
    M, K = xq.shape
    N = codes.shape[0]
    sd = torch.empty(scales.size + scale_offset, dtype=torch.bfloat16, device="cuda")
    sd = sd[scale_offset:].view(N, K // 32).copy_(dev_bf16(scales))
    band = torch.full((M * N + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = band[32:32 + M * N].view(M, N)
    got = api.w4a8_linear(torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), dev_u32(codes), sd, y=y)
    torch.cuda.synchronize()
    ref = decode.w4a8_linear(xq, xs, codes, scales)
    mag = decode.w4a8_magnitude(xq, xs, codes, scales)
    err = np.abs(host_f64(got) - ref)
    assert (err <= np.abs(ref) * HALF_BF16 + mag * (K // 32 + 4) * 2.0 ** -24 * 1.01).all()
    assert (band[:32] == 3).all() and (band[32 + M * N:] == 3).all()


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130])
@pytest.mark.parametrize("N,K", [(256, 256), (1, 32), (7, 64), (40, 352), (129, 1024), (72, 4096)])
def test_linear(M, N, K):
    check_linear(*linear_case(M, N, K, M * N + K))


@pytest.mark.parametrize("M,N,K", [(1, 14336, 4096), (16, 1500, 2816), (3, 17, 32 * 61), (300, 1024, 704),
                                   (509, 300, 2816), (1000, 130, 96), (5, 2000, 8192), (12, 64, 32768),
                                   (16, 64, 65536)])
def test_linear_wider(M, N, K):
    check_linear(*linear_case(M, N, K, 11))


@pytest.mark.parametrize("M,N,K,off", [(900, 5632, 1024, 0), (1025, 3584, 1088, 0), (900, 5632, 1024, 1),
                                       (509, 8192, 448, 0), (300, 16384, 832, 0), (64, 14336, 4096, 0), (64, 14336, 4096, 1),
                                       (385, 9472, 64 * 17, 0), (257, 9472, 2048, 0)])
def test_linear_many_rows(M, N, K, off):
    xq, xs, codes, scales = linear_case(M, N, K, 5)
    xs[7] = np.nan
    assert api.w4_workspace_bytes(_lib.W4_OP_LINEAR_8, M, N, K, 1, 1) >= M * K * 2      # the converted rows
    sd = torch.empty(scales.size + off, dtype=torch.bfloat16, device="cuda")
    sd = sd[off:].view(N, K // 32).copy_(dev_bf16(scales))
    y = host_f64(api.w4a8_linear(torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), dev_u32(codes), sd))
    assert np.isnan(y[7]).all()
    keep = np.delete(np.arange(M), 7)
    w = np.abs(decode.row_values(*_rows_of(codes, scales)))
    mag = (np.abs(xq[keep].astype(np.float64)) @ w.T) * np.abs(xs[keep].astype(np.float64))[:, None]
    ref = decode.w4a8_linear(xq[keep], xs[keep], codes, scales)
    assert (np.abs(y[keep] - ref) <= np.abs(ref) * HALF_BF16 + mag * (K / 16) * 2.0 ** -23).all()


def _rows_of(codes, scales):
    q = np.zeros((codes.shape[0], codes.shape[1] * 8), np.int64)
    for j in range(8):
        q[:, j::8] = ((codes >> np.uint32(4 * j)) & np.uint32(15)).astype(np.int64) - 8
    return q, scales


@pytest.mark.parametrize("M", [4, 40, 200])
def test_linear_largest_group_sums(M):
    check_linear(*linear_case(M, 96, 1024, 3, peak=True))


@pytest.mark.parametrize("off", [1, 2, 4])
def test_linear_scales_at_any_even_address(off):
    check_linear(*linear_case(9, 80, 512, 21), scale_offset=off)


def test_linear_nan_scale_of_a_row_reaches_that_row_alone():
    xq, xs, codes, scales = linear_case(6, 64, 512, 4)
    xs[2] = np.nan
    y = host_f64(api.w4a8_linear(torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), dev_u32(codes),
                                 dev_bf16(scales)))
    assert np.isnan(y[2]).all() and np.isfinite(np.delete(y, 2, axis=0)).all()


def test_linear_same_bits_every_time():
    xq, xs, codes, scales = linear_case(16, 3000, 4096, 8)
    a = [torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), dev_u32(codes), dev_bf16(scales)]
    first = api.w4a8_linear(*a).clone()
    for _ in range(5):
        assert torch.equal(api.w4a8_linear(*a), first)
