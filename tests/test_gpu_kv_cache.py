"""GPU parity of the paged key/value cache: writes and reads bit for bit, attention within derived
bounds of the float64 oracle.

Attention's bound, per element, with P = sum p |v| over the sequence and z = scale * max sum |q k|:
  * out is rounded to bf16 once: 2^-8 of the value;
  * the weights p and the scaled values each enter the product with at most one rounding to 11 bits
    (half a step 2^-11 relative each): (2^-11 + 2^-11) P, doubled for the sum of weights not
    sharing the weights' roundings: 2^-9 P covers both;
  * scores are float32 dot products: off by (D + 16) 2^-24 z, which moves a weight by twice that;
  * a weight is held in fp16 as 2^6 p, p being relative to a score some token of its warp had, so the
    weights sum to 1 at least: below the normal range a rounding is half of 2^-24, which is 2^-31 of
    the sum per token, 2^-31 sum |v| in all.
"""
import numpy as np
import pytest
import torch

from oracle import bf16, decode
from w4a16_group_quantized_w4_b200 import _lib, api
from tests._util import dev_bf16, host_bf16_bits, host_f64, host_u32

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "int8", "int4"]


def rows(r, n, heads, dim):
    return bf16.from_f64(r.randn(n, heads, dim) * np.exp(0.5 * r.randn(heads, dim)))


def host_codes(t, kind):
    return host_bf16_bits(t) if kind == "bf16" else host_u32(t) if kind == "int4" else t.cpu().numpy()


def stored(x, kind):
    """x bits [n, heads, dim] -> what the cache holds for it: (codes, scale bits or None)."""
    if kind == "bf16":
        return x, None
    n, heads, dim = x.shape
    q, s = decode.quantise_rows(x.reshape(-1, dim), kind)
    s = s.reshape(n, heads, dim // 32)
    if kind == "int4":
        return decode.pack_l1(q).reshape(n, heads, dim // 8), s
    return q.astype(np.int8).reshape(n, heads, dim), s


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,heads,dim,page", [(1, 1, 32, 1), (5, 2, 64, 16), (37, 3, 96, 7), (64, 8, 128, 32),
                                              (130, 2, 256, 24), (9, 20, 192, 64), (3, 1, 1024, 2)])
def test_write_then_read(kind, T, heads, dim, page):
    r = np.random.RandomState(T + dim)
    pages = T // page + 3
    cache = api.KVCache(pages, heads, page, dim, kind)
    for t in (cache.k, cache.v):                      # a pattern to find untouched rows by
        t.view(torch.uint8).fill_(0x5A)
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[[1, 3]] = -1
    k, v = rows(r, T, heads, dim), rows(r, T, heads, dim)
    sd = torch.from_numpy(slots).cuda()
    # columns of a wider row: a query part in front, keys, values
    wide = torch.randn((T, heads * dim * 2 + 8), device="cuda").to(torch.bfloat16)
    kd = wide[:, 8:8 + heads * dim].unflatten(1, (heads, dim))
    vd = wide[:, 8 + heads * dim:].unflatten(1, (heads, dim))
    kd.copy_(dev_bf16(k))
    vd.copy_(dev_bf16(v))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(kd, vd, sd, dev_status=st)
    keep = slots >= 0
    at = slots[keep] // page, slots[keep] % page
    back = cache.read(sd, dev_status=st)
    assert st.item() == 0
    for x, buf, sc, out in ((k, cache.k, cache.k_scales, back[0]), (v, cache.v, cache.v_scales, back[1])):
        codes, scales = stored(x[keep], kind)
        got = host_codes(buf, kind)
        assert np.array_equal(got[at[0], :, at[1]], codes)
        touched = np.zeros((pages, page), bool)
        touched[at] = True
        left = got.transpose(0, 2, 1, 3)[~touched]
        assert (np.ascontiguousarray(left).view(np.uint8) == 0x5A).all()
        out = host_bf16_bits(out)
        assert not out[~keep].any()
        if kind == "bf16":
            assert np.array_equal(out[keep], codes)
            continue
        gs = host_bf16_bits(sc)
        assert np.array_equal(gs[at[0], :, at[1]], scales)
        assert not gs.transpose(0, 2, 1, 3)[~touched].any()
        q, s = decode.quantise_rows(x[keep].reshape(-1, dim), kind)
        assert np.array_equal(out[keep], bf16.from_f64(decode.row_values(q, s)).reshape(out[keep].shape))


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_groups_of_every_size(kind):
    """Groups over the whole exponent range, subnormal steps, zeros, infinities and NaN."""
    r = np.random.RandomState(2)
    T, dim = 300, 64
    x = r.randn(T, 1, dim) * 2.0 ** r.randint(-133, 127, (T, 1, 1))
    x = bf16.from_f64(np.clip(x, -3e38, 3e38))
    x[7, 0, :32] = 0
    x[8, 0, 3], x[9, 0, 40], x[10, 0, 0] = 0x7F80, 0xFF80, 0x7FC1
    x[11, 0, :32] = 1                                  # the smallest subnormal
    x[12, 0, 32:] = 0x8000                             # minus zero
    cache = api.KVCache(T, 1, 1, dim, kind)
    d = dev_bf16(x)
    cache.write(d, d, torch.arange(T, device="cuda"))
    codes, scales = stored(x, kind)
    assert np.array_equal(host_codes(cache.k, kind)[:, :, 0], codes)
    assert np.array_equal(host_bf16_bits(cache.v_scales)[:, :, 0], scales)
    back = host_f64(cache.read(torch.arange(T, device="cuda"))[0])
    assert np.isnan(back[8, 0, :32]).all() and np.isnan(back[9, 0, 32:]).all() and np.isfinite(back[9, 0, :32]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_slots_past_the_cache_are_reported_and_dropped(kind):
    cache = api.KVCache(3, 2, 8, 64, kind)
    before = cache.k.clone()
    k = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([24, 1 << 40, -5], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(k, k, slots, dev_status=st)
    assert st.item() == 1 and torch.equal(cache.k, before)
    st.zero_()
    a, b = cache.read(slots, dev_status=st)
    assert st.item() == 1 and not a.any() and not b.any()


# ------------------------------------------------------------------------------- attention
class Seqs:
    """Sequences of given lengths in a paged cache with shuffled pages, and their float64 rows."""

    def __init__(self, lens, heads, dim, page, kind, seed, junk=True, size=1.0, spread=0):
        r = np.random.RandomState(seed)
        self.lens, self.heads, self.dim, self.kind = lens, heads, dim, kind
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        self.cache = api.KVCache(pages, heads, page, dim, kind)
        if junk:                       # what lies in unused places must not matter: NaN patterns
            if kind == "bf16":
                self.cache.k.fill_(float("nan"))
                self.cache.v.fill_(float("nan"))
            else:
                for t in (self.cache.k, self.cache.v):
                    t.view(torch.uint8).fill_(0x77)
                self.cache.k_scales.fill_(float("nan"))
                self.cache.v_scales.fill_(float("inf"))
        order = r.permutation(pages)
        self.table = np.full((len(lens), max(1, max(need)) + 1), -1, np.int32)
        at = 0
        self.k, self.v = [], []
        slots, ks, vs = [], [], []
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            pos = np.arange(n)
            slots.append(self.table[b, pos // page].astype(np.int64) * page + pos % page)
            ks.append(rows(r, n, heads, dim))
            each = 2.0 ** np.random.RandomState(n).randint(-spread, spread + 1, (n, 1, 1))
            vs.append(bf16.from_f64(size * each * bf16.to_f64(rows(r, n, heads, dim))))
        slots = np.concatenate(slots)
        k, v = np.concatenate(ks), np.concatenate(vs)
        if len(slots):
            self.cache.write(dev_bf16(k), dev_bf16(v), torch.from_numpy(slots).cuda())
        if kind == "bf16":
            fk, fv = bf16.to_f64(k), bf16.to_f64(v)
        else:                          # codes and scales were checked above; their exact products
            fk, fv = (self._values(c, s, slots, page) for c, s in
                      ((self.cache.k, self.cache.k_scales), (self.cache.v, self.cache.v_scales)))
        cut = np.cumsum(lens)[:-1]
        self.k, self.v = np.split(fk, cut), np.split(fv, cut)
        self.table_d = torch.from_numpy(self.table).cuda()
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def _values(self, codes, scales, slots, page):
        c = host_codes(codes, self.kind)[slots // page, :, slots % page]
        s = bf16.to_f64(host_bf16_bits(scales)[slots // page, :, slots % page])
        if self.kind == "int4":
            q = np.zeros(c.shape[:-1] + (c.shape[-1] * 8,))
            for j in range(8):
                q[..., j::8] = ((c >> np.uint32(4 * j)) & np.uint32(15)).astype(np.float64) - 8
            c = q
        return c.astype(np.float64) * np.repeat(s, 32, axis=-1)

    def check(self, q_heads, seed=0, scale=None, softcap=0.0, window=0, strided=False, q=None, floor=0.0):
        r = np.random.RandomState(seed)
        B = len(self.lens)
        q = bf16.from_f64(r.randn(B, q_heads, self.dim)) if q is None else q
        qd = dev_bf16(q)
        if strided:
            wide = torch.zeros((B, (q_heads + 2) * self.dim), dtype=torch.bfloat16, device="cuda")
            qd = wide[:, :q_heads * self.dim].unflatten(1, (q_heads, self.dim)).copy_(qd)
        band = torch.full((B + 2, q_heads, self.dim), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((B, q_heads), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = self.cache.attend(qd, self.table_d, self.lens_d, scale=scale, softcap=softcap, window=window,
                                out=band[1:-1], lse=lse, dev_status=st)
        assert st.item() == 0 and (band[0] == 9).all() and (band[-1] == 9).all()
        got, lse = host_f64(out), lse.cpu().numpy().astype(np.float64)
        scale = self.dim ** -0.5 if scale is None else scale
        qf = bf16.to_f64(q)
        G = q_heads // self.heads
        for b in range(B):
            for h in range(q_heads):
                ref, ref_lse, mag, peak, vsum = decode.attend(qf[b, h], self.k[b][:, h // G], self.v[b][:, h // G], scale,
                                                        softcap, window)
                dz = (self.dim + 16) * 2.0 ** -24 * abs(scale) * peak + 2.0 ** -20 * max(1.0, softcap)
                tol = np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -9 + 2 * dz) + 2.0 ** -31 * vsum
                if floor:
                    tol = tol + floor * np.abs(self.v[b][:, h // G]).max()
                assert (np.abs(got[b, h] - ref) <= tol).all(), (b, h, np.abs(got[b, h] - ref).max())
                if self.lens[b]:
                    assert abs(lse[b, h] - ref_lse) <= 2.0 ** -11 + 2 * dz + abs(ref_lse) * 2.0 ** -23
                else:
                    assert lse[b, h] == -np.inf
        return out


LENS = [1, 0, 15, 16, 17, 63, 64, 65, 0, 130, 257, 2]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_attend(kind, dim, page):
    Seqs(LENS, 2, dim, page, kind, dim + page).check(8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,q_heads", [(1, 1), (3, 3), (2, 10), (1, 7), (4, 32), (1, 9), (2, 32), (1, 40), (5, 60)])
def test_head_layouts(kind, heads, q_heads):
    Seqs([33, 1, 200], heads, 128, 32, kind, heads).check(q_heads, strided=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 16, 50, 1000])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_window_and_softcap(kind, window, softcap):
    Seqs([0, 1, 15, 49, 50, 51, 64, 113, 300], 2, 64, 16, kind, window).check(6, softcap=softcap, window=window)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,dim,page", [([5000], 128, 16), ([9001, 3, 700], 64, 64), ([2500], 256, 7),
                                           ([4097, 4096], 192, 128)])
def test_long_sequences_split_and_joined(kind, lens, dim, page):
    Seqs(lens, 1, dim, page, kind, 5).check(4, scale=0.2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,q_heads,lens,page", [(1, 9, [3000], 16), (1, 16, [1, 2049, 0, 700], 7), (2, 40, [4100, 65], 48),
                                                     (1, 33, [1800], 32)])
def test_many_heads_over_long_sequences(kind, dim, heads, q_heads, lens, page):
    """Items of 16 heads, cut and joined, the last of them with fewer."""
    Seqs(lens, heads, dim, page, kind, q_heads).check(q_heads, scale=0.2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [192, 256])
def test_many_heads_of_wide_rows(kind, dim):
    Seqs([1500, 90], 1, dim, 16, kind, dim).check(20, scale=0.2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,softcap", [(700, 0.0), (1999, 3.0), (2049, 0.0)])
@pytest.mark.parametrize("q_heads", [4, 12])
def test_window_over_long_sequences(kind, window, softcap, q_heads):
    Seqs([2000, 5, 3333, 2049], 1, 128, 16, kind, 9).check(q_heads, softcap=softcap, window=window)


# tables of 8 units over 600 items, and of 20 units over 2500: a block takes an item whole
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,longest,heads,q_heads,dim", [(150, 496, 4, 4, 64), (75, 480, 8, 80, 64), (320, 1264, 8, 8, 64)])
def test_items_taken_whole(kind, B, longest, heads, q_heads, dim):
    r = np.random.RandomState(B)
    lens = [int(n) for n in np.minimum(longest, 2 ** r.uniform(0, np.log2(longest), B))]
    lens[3], lens[5] = longest, 0
    Seqs(lens, heads, dim, 16, kind, 4).check(q_heads)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    r = np.random.RandomState(8)
    lens = [int(n) for n in r.randint(0, 90, 300)]
    Seqs(lens, 2, 64, 16, kind, 4).check(4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [3.0, -0.5, 1e-4])
def test_sharp_and_flat_softmax(kind, scale):
    Seqs([700, 64], 2, 128, 32, kind, 6).check(4, scale=scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
def test_values_of_unlike_sizes(kind, size):
    Seqs([200, 31], 2, 64, 16, kind, 7, size=size).check(4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.125, 4.0])
def test_tokens_of_unlike_sizes(kind, scale):
    """Tokens whose values lie 2^20 apart: a large one of no weight must not cost a small one its bits.  Below
    the normal range scaled fp16 values are off by 2^-21 (int8) or 2^-20 (int4) of the largest scale, and a scale
    is at most the largest value of its group over 127 or 7: 2^-27 or 2^-22 of the largest value."""
    floor = {"bf16": 0.0, "int8": 2.0 ** -27, "int4": 2.0 ** -22}[kind]
    Seqs([200, 31, 1500], 2, 64, 16, kind, 7, spread=10).check(4, scale=scale, floor=floor)


@pytest.mark.parametrize("kind", KINDS)
def test_queries_of_unlike_sizes(kind):
    r = np.random.RandomState(3)
    q = bf16.from_f64(r.randn(2, 8, 64) * 2.0 ** r.randint(-8, 3, (2, 8, 64)) * 2.0 ** r.randint(-40, 3, (2, 8, 1)))
    Seqs([90, 700], 2, 64, 16, kind, 3).check(8, q=q)


def test_lengths_and_pages_out_of_range_are_reported():
    s = Seqs([40, 40, 40], 1, 64, 16, "bf16", 1)
    q = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    good = s.cache.attend(q, s.table_d, s.lens_d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = s.lens_d.clone()
    lens[1] = -3
    out = s.cache.attend(q, s.table_d, lens, dev_status=st)
    assert st.item() == 1 and not out[1].any() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    # a page outside the cache: its 16 tokens are left out
    st.zero_()
    table = s.table_d.clone()
    table[2, 1] = 1 << 30
    out = s.cache.attend(q, table, s.lens_d, dev_status=st)
    assert st.item() == 1 and torch.equal(out[0], good[0])
    keep = np.r_[0:16, 32:40]
    for h in range(2):
        ref, _, mag, *_ = decode.attend(host_f64(q)[2, h], s.k[2][keep, 0], s.v[2][keep, 0], 0.125)
        assert (np.abs(host_f64(out)[2, h] - ref) <= np.abs(ref) * 2.0 ** -8 + mag * 2.0 ** -8).all()
    # a length past the table: cut to it (its last column names no page, so those tokens fall out too)
    st.zero_()
    lens = s.lens_d.clone()
    lens[0] = 1 << 20
    out = s.cache.attend(q, s.table_d, lens, dev_status=st)
    assert st.item() == 1 and torch.equal(out[1], good[1])


@pytest.mark.parametrize("kind", KINDS)
def test_same_bits_every_time_and_on_another_stream(kind):
    s = Seqs([3000, 5, 900], 2, 128, 16, kind, 2)
    q = torch.randn((3, 8, 128), device="cuda").to(torch.bfloat16)
    first = s.cache.attend(q, s.table_d, s.lens_d).clone()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    outs = [s.cache.attend(q, s.table_d, s.lens_d, stream=other) for _ in range(3)]
    outs += [s.cache.attend(q, s.table_d, s.lens_d) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_output_beside_the_queries_but_not_over_them():
    s = Seqs([40, 300], 2, 64, 16, "int8", 3)
    rows = torch.randn((4, 4, 64), device="cuda").to(torch.bfloat16)
    want = s.cache.attend(rows[:2].clone(), s.table_d, s.lens_d)
    with pytest.raises(_lib.W4Error):
        s.cache.attend(rows[:2], s.table_d, s.lens_d, out=rows[1:3])
    got = s.cache.attend(rows[:2], s.table_d, s.lens_d, out=rows[2:])
    assert torch.equal(got, want)
    other = s.cache.attend(rows[2:], s.table_d, s.lens_d, out=rows[:2])
    assert other.data_ptr() == rows.data_ptr()


@pytest.mark.parametrize("kind", KINDS)
def test_two_graphs_replayed_side_by_side(kind):
    """A write and an attention captured twice; the graphs replay on two streams at once, with new
    contents in their static inputs."""
    seqs = [Seqs([2100, 17], 2, 128, 16, kind, n) for n in (1, 2)]
    sides = []
    for s in seqs:
        q = torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16)
        k = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
        slots = s.cache.slots(s.table_d, s.lens_d - 1)
        s.cache.write(k, k, slots)
        s.cache.attend(q, s.table_d, s.lens_d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.cache.write(k, k, slots)
            out = s.cache.attend(q, s.table_d, s.lens_d)
        sides.append((g, q, k, out, s))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for g, q, k, out, s in sides:
        q.copy_(torch.randn((2, 8, 128), device="cuda"))
        k.copy_(torch.randn((2, 2, 128), device="cuda"))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (g, *_rest) in zip(streams, sides):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for g, q, k, out, s in sides:
        assert torch.equal(out, s.cache.attend(q, s.table_d, s.lens_d))


@pytest.mark.parametrize("kind", KINDS)
def test_rows_past_2_31_bytes(kind):
    """Offsets of the last pages of a large cache pass 32 bits (in elements for the codes)."""
    dim, heads, page = 256, 8, 64
    per_page = heads * page * dim
    pages = (1 << 32) // per_page + 3
    cache = api.KVCache(pages, heads, page, dim, kind)
    r = np.random.RandomState(1)
    n = 70
    k, v = rows(r, n, heads, dim), rows(r, n, heads, dim)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = table.long()[0, pos // page] * page + pos % page
    cache.write(dev_bf16(k), dev_bf16(v), slots)
    a, b = cache.read(slots)
    q = bf16.from_f64(r.randn(1, heads, dim))
    out = host_f64(cache.attend(dev_bf16(q), table, torch.tensor([n], dtype=torch.int32, device="cuda")))
    small = api.KVCache(2, heads, page, dim, kind)
    st = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    small.write(dev_bf16(k), dev_bf16(v), pos)
    c, d = small.read(pos)
    assert torch.equal(a, c) and torch.equal(b, d)
    want = host_f64(small.attend(dev_bf16(q), st, torch.tensor([n], dtype=torch.int32, device="cuda")))
    assert np.array_equal(out, want)
    del cache
    torch.cuda.empty_cache()
