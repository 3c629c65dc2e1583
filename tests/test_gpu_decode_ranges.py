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
from tests.test_gpu_kv_cache import KINDS
from tests.test_gpu_rms_add import check_linear, linear_case

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


class Filled:
    """Sequences of given lengths over rows that the caller makes: k, v bf16 bits [sum of lens, heads, dim]."""

    def __init__(self, lens, k, v, page, kind, seed=0):
        r = np.random.RandomState(seed)
        _, heads, dim = k.shape
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 1
        order = r.permutation(pages)
        table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        slots, at = [], 0
        for b, n in enumerate(lens):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            pos = np.arange(n)
            slots.append(table[b, pos // page].astype(np.int64) * page + pos % page)
        slots = np.concatenate(slots)
        self.lens, self.heads, self.dim, self.kind = lens, heads, dim, kind
        self.cache = api.KVCache(pages, heads, page, dim, kind)
        self.cache.write(dev_bf16(k), dev_bf16(v), torch.from_numpy(slots).cuda())
        cut = np.cumsum(lens)[:-1]
        self.k, self.v, self.ks = [], [], []
        for x, out in ((k, self.k), (v, self.v)):
            if kind == "bf16":
                f, s = bf16.to_f64(x), np.zeros((len(x), heads, dim))
            else:
                q, sb = decode.quantise_rows(x.reshape(-1, dim), kind)
                f = decode.row_values(q, sb).reshape(x.shape)
                s = np.repeat(bf16.to_f64(sb), 32, axis=1).reshape(x.shape)
            out.extend(np.split(f, cut))
            if out is self.k:
                self.ks = np.split(s, cut)               # a key element's scale (0: none)
        self.table = torch.from_numpy(table).cuda()
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def attend(self, q, **kw):
        lse = torch.empty(q.shape[:2], device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = self.cache.attend(dev_bf16(q), self.table, self.lens_d, lse=lse, dev_status=st, **kw)
        assert st.item() == 0
        return host_f64(out), lse.cpu().numpy().astype(np.float64)

    def check(self, q, scale=None, softcap=0.0, window=0):
        """Scores: a group's products and its bias (128 scales an element, int8; 8, int4) are summed in float32 in
        at most dim / 16 + dim / 32 + 5 steps, each off by 2^-22 of the magnitudes in it (a tensor-core step may
        cut off where float32 would round); a cap adds 2^-20 of the score, or, up to 64, 2^-21 of
        itself (2^x within 2^-22, a reciprocal within 2^-23)."""
        out, lse = self.attend(q, scale=scale, softcap=softcap, window=window)
        scale = self.dim ** -0.5 if scale is None else scale
        qf, G = bf16.to_f64(q), q.shape[1] // self.heads
        bias = {"bf16": 0.0, "int8": 128.0, "int4": 8.0}[self.kind]
        steps = self.dim / 16 + self.dim / 32 + 5
        for b, n in enumerate(self.lens):
            seen = slice(max(0, n - window) if window else 0, n)
            for h in range(q.shape[1]):
                k, v, ks = (x[b][seen, h // G] for x in (self.k, self.v, self.ks))
                ref, ref_lse, mag, _, vsum = decode.attend(qf[b, h], k, v, scale, softcap)
                if n == 0:
                    assert lse[b, h] == -np.inf and not out[b, h].any()
                    continue
                size = np.max((np.abs(k) + 2 * bias * ks) @ np.abs(qf[b, h])) * abs(scale)
                dz = steps * 2.0 ** -22 * size + 2.0 ** -22
                if softcap:
                    dz += 2.0 ** -21 * softcap if softcap <= 64 else 2.0 ** -20 * np.abs(k @ qf[b, h]).max() * abs(scale)
                assert abs(lse[b, h] - ref_lse) <= dz + 2.0 ** -17 + abs(ref_lse) * 2.0 ** -22, (b, h, lse[b, h] - ref_lse, dz)
                tol = np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -9 + 2 * dz) + 2.0 ** -31 * vsum
                assert (np.abs(out[b, h] - ref) <= tol).all(), (b, h, np.abs(out[b, h] - ref).max())


def normal(r, *shape):
    return r.randn(*shape) * np.exp(0.5 * r.randn(*shape[1:]))


LENS = [1, 0, 17, 130, 1500]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("softcap", [1e-3, 50.0, 64.0, 65.0, 300.0, 1e4, 1e6, 1e8, 1e20, 1e38, 3.4e38])
def test_caps_of_every_size(kind, softcap):
    """Scores far below the cap come out as they went in, to float32's last places."""
    r = np.random.RandomState(3)
    k, v = (bf16.from_f64(normal(r, sum(LENS), 2, 64)) for _ in range(2))
    Filled(LENS, k, v, 16, kind).check(bf16.from_f64(r.randn(len(LENS), 6, 64)), softcap=softcap)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,q_heads", [(128, 12), (256, 4)])
@pytest.mark.parametrize("scale", [1.0, 6.0])
def test_scores_around_a_large_cap(kind, dim, q_heads, scale):
    """Scores on both sides of half the cap, where the way to tanh changes, and far past it."""
    r = np.random.RandomState(4)
    k, v = (bf16.from_f64(normal(r, 700, 1, dim)) for _ in range(2))
    Filled([650, 50], k, v, 16, kind).check(bf16.from_f64(r.randn(2, q_heads, dim)), scale=scale, softcap=100.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 24, 64])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_large_caps_over_pages_and_windows(kind, page, window):
    r = np.random.RandomState(page)
    lens = [0, 1, 70, 333, 64]
    k, v = (bf16.from_f64(normal(r, sum(lens), 2, 192)) for _ in range(2))
    Filled(lens, k, v, page, kind).check(bf16.from_f64(r.randn(len(lens), 6, 192)), softcap=1e5, window=window)


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("dim,q_heads", [(64, 4), (128, 12), (256, 3)])
def test_values_at_the_end_of_the_range(kind, dim, q_heads):
    """Groups whose scales are among the largest that finite rows have (2^120, int8; 2^125, int4), among smaller ones;
    items that a block holds whole, and cut ones."""
    r = np.random.RandomState(dim)
    lens = [1, 40, 0, 3000]
    k = bf16.from_f64(normal(r, sum(lens), 1, dim))
    v = r.uniform(0.5, 1.0, (sum(lens), 1, dim)) * r.choice([-1, 1], (sum(lens), 1, dim))
    v *= 3.3e38 * 2.0 ** -r.randint(0, 6, (sum(lens), 1, dim // 32)).repeat(32, axis=2)
    Filled(lens, k, bf16.from_f64(v), 16, kind).check(bf16.from_f64(r.randn(len(lens), q_heads, dim)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,q_heads", [(64, 4), (128, 12)])
@pytest.mark.parametrize("size", [-113, -105, -60, 90, 100, 110, 119])
def test_ordinary_scores_of_large_and_small_keys(kind, dim, q_heads, size):
    """Keys of about 2^size under queries of about 2^-size: a sum in front of the last factor may leave float32's
    range although no score does."""
    r = np.random.RandomState(dim)
    lens = [1, 33, 700]
    k = bf16.from_f64(np.clip(normal(r, sum(lens), 1, dim) * 2.0 ** size, -3e38, 3e38))
    v = bf16.from_f64(normal(r, sum(lens), 1, dim))
    q = r.randn(len(lens), q_heads, dim) * 2.0 ** -size
    Filled(lens, k, v, 16, kind).check(bf16.from_f64(np.clip(q, -3e38, 3e38)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [-126, -100, 0, 110])
def test_heads_of_unlike_sizes_beside_one_another(kind, size):
    """Query heads of one item whose elements lie 2^20 to 2^120 apart."""
    r = np.random.RandomState(9)
    lens = [40, 200]
    k, v = (bf16.from_f64(normal(r, sum(lens), 1, 128) * s) for s in (2.0 ** -115, 1.0))
    q = r.randn(2, 20, 128) * 2.0 ** np.tile([115.0, 116, 117, 95, size], 4)[:, None]
    Filled(lens, k, v, 16, kind).check(bf16.from_f64(np.clip(q, -3e38, 3e38)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,heads,q_heads", [(64, 2, 4), (128, 2, 24)])
def test_nan_reaches_the_output_and_lse_of_its_heads_alone(kind, dim, heads, q_heads):
    """A NaN query, and a cached key that held an infinity (a group of NaN; an infinity in a bf16 cache), in a short
    sequence and in a long one that is cut: out and lse are NaN, not the -infinity of an empty sequence."""
    r = np.random.RandomState(dim)
    lens = [20, 3000, 1, 20, 3000, 0]
    G = q_heads // heads
    k, v = (bf16.from_f64(normal(r, sum(lens), heads, dim)) for _ in range(2))
    q = bf16.from_f64(r.randn(len(lens), q_heads, dim))
    clean = Filled(lens, k, v, 16, kind).attend(q)
    start = np.cumsum([0] + lens)
    for b, token in ((0, 7), (1, 1700)):
        k[start[b] + token, 1, dim - 3] = 0x7FC0 if kind == "bf16" else 0x7F80
    q[3, 1, 5], q[4, G + 1, 0] = 0x7FC0, 0xFFC1
    out, lse = Filled(lens, k, v, 16, kind).attend(q)
    bad = np.zeros(lse.shape, bool)
    bad[0, G:] = bad[1, G:] = True
    bad[3, 1] = bad[4, G + 1] = True
    assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
    # (the others' references may be raised at other tokens: weights within fp16's rounding)
    assert (np.abs(out - clean[0])[~bad] <= 2.0 ** -7 * np.abs(clean[0][~bad]) + 2.0 ** -8 * np.abs(bf16.to_f64(v)).max()).all()
    both = ~bad & (lse > -np.inf)
    assert (np.abs(lse[both] - clean[1][both]) <= 2.0 ** -16).all()
    assert np.isneginf(lse[5]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_nan_values_leave_lse_alone(kind):
    r = np.random.RandomState(6)
    lens = [20, 3000]
    k, v = (bf16.from_f64(normal(r, sum(lens), 1, 64)) for _ in range(2))
    q = bf16.from_f64(r.randn(2, 4, 64))
    clean = Filled(lens, k, v, 16, kind).attend(q)
    size = np.abs(bf16.to_f64(v)).max()
    v[[3, 20 + 1700], 0, 40] = 0x7FC0
    out, lse = Filled(lens, k, v, 16, kind).attend(q)
    gone = slice(40, 41) if kind == "bf16" else slice(32, 64)
    assert np.isnan(out[:, :, gone]).all() and np.array_equal(lse, clean[1])
    assert (np.abs(out - clean[0])[:, :, :32] <= 2.0 ** -7 * np.abs(clean[0][:, :, :32]) + 2.0 ** -8 * size).all()


@pytest.mark.parametrize("T,H,residual", [(1, 64, False), (3, 512, True), (300, 2816, True), (2, 32768, False), (2, 8200, True)])
def test_rows_without_eps(T, H, residual):
    """eps = 0: a row of zeros gives zeros (scale 0, codes 0); rows whose squares are below float32's range are
    normalised all the same.  Bounds as in test_gpu_rms_add.py: the sum is at most H / 8 + 8 roundings long
    there, (H / 32 + 16) in the way tiny rows take, and a subnormal product h w is off by 2^-150, divided by
    the root mean square like the rest."""
    r = np.random.RandomState(H)
    size = 2.0 ** r.randint(-120, 50, (T, 1))
    size[0] = 2.0 ** -100
    x = size * r.randn(T, H)
    res = bf16.from_f64(size * r.randn(T, H)) if residual else None
    x = bf16.from_f64(x)
    w = bf16.from_f64(1 + 0.3 * r.randn(H))
    if T > 2:
        x[1] = 0
        if residual:
            res[1] = 0
    dres = None if res is None else dev_bf16(res)
    y, h = api.w4_rms_add(dev_bf16(x), dres, dev_bf16(w), eps=0.0)
    q, qs, h2 = api.w4_rms_add_q8(dev_bf16(x), dres, dev_bf16(w), eps=0.0)
    y, q, qs = host_f64(y), q.cpu().numpy().astype(np.float64), qs.cpu().numpy().astype(np.float64)
    hb = host_bf16_bits(h)
    assert np.array_equal(hb, host_bf16_bits(h2))
    zero = ~(hb & 0x7FFF).any(axis=1)
    assert zero.any() == (T > 2)
    assert not y[zero].any() and not q[zero].any() and not qs[zero].any()
    with np.errstate(invalid="ignore"):
        h_ref, y_ref = decode.rms_add(x, res, w, 0.0)
    assert np.array_equal(hb, h_ref)
    y, q, qs, y_ref = (t[~zero] for t in (y, q, qs, y_ref))
    off = 2.0 ** -150 / np.sqrt(np.mean(bf16.to_f64(h_ref)[~zero] ** 2, axis=1, keepdims=True))
    rel = (H / 8 + 16) * 2.0 ** -24 * 1.01
    assert (np.abs(y - y_ref) <= np.abs(y_ref) * (2.0 ** -8 + rel) + 1.01 * off).all()
    s_ref = np.abs(y_ref).max(axis=1) / 127
    assert (np.abs(qs - s_ref) <= s_ref * rel + 1.01 * off[:, 0] / 127).all()
    assert (np.abs(q - y_ref / s_ref[:, None]) <= 0.5 + 127 * 3 * rel + 2 * off / s_ref[:, None]).all()


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-38, 1e-33, 1e-28, 1e-26])
@pytest.mark.parametrize("T,H", [(5, 256), (4, 2816), (301, 2816), (3, 16392)])
def test_tiny_rows_beside_a_tiny_eps(eps, T, H):
    """Rows far below, about and above the root of eps, without a weight, the residual updated in place."""
    r = np.random.RandomState(T)
    root = np.sqrt(np.float32(max(eps, 1e-42)).astype(np.float64))
    size = root * 2.0 ** r.randint(-20, 21, (T, 1))
    x, res = (bf16.from_f64(size * r.randn(T, H)) for _ in range(2))
    e = float(np.float32(eps))
    h_ref, y_ref = decode.rms_add(x, res, None, e)
    rel = (H / 8 + 16) * 2.0 ** -24 * 1.01
    buf = dev_bf16(res)
    y, h = api.w4_rms_add(dev_bf16(x), buf, eps=e, h=buf)
    assert h is buf and np.array_equal(host_bf16_bits(h), h_ref)
    assert (np.abs(host_f64(y) - y_ref) <= np.abs(y_ref) * (2.0 ** -8 + rel)).all()
    buf = dev_bf16(res)
    q, qs, h = api.w4_rms_add_q8(dev_bf16(x), buf, eps=e, h=buf)
    assert np.array_equal(host_bf16_bits(h), h_ref)
    s_ref = np.abs(y_ref).max(axis=1) / 127
    assert (np.abs(qs.cpu().numpy() - s_ref) <= s_ref * rel).all()
    assert (np.abs(q.cpu().numpy() - y_ref / s_ref[:, None]) <= 0.5 + 127 * 3 * rel).all()


@pytest.mark.parametrize("M,N,K", [(17, 300, 8192), (32, 1024, 5120), (31, 129, 32 * 161), (17, 19000, 4928), (20, 5, 4896)])
def test_linear_of_17_to_32_rows_too_long_for_shared_memory(M, N, K):
    """The tiled kernel with 32 tokens a tile: K split and whole, scales by TMA and not."""
    check_linear(*linear_case(M, N, K, M + N))
