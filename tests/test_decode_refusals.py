"""Host-side refusals of the norm, 8-bit linear and cache entry points (CPU only: every check comes
before any CUDA call, so the pointers are never followed)."""
import ctypes as C

import pytest
import torch

from w4a16_group_quantized_w4_b200 import _lib, api

P = 4096            # a well aligned, never dereferenced address
BAD, UNSUP, WS = _lib.W4_ERR_INVALID_ARG, _lib.W4_ERR_UNSUPPORTED, _lib.W4_ERR_WORKSPACE


def rms(lib, q8=False, x=P, res=P, w=P, T=4, H=64, eps=1e-6, h=P, out=P, qs=P):
    if q8:
        return lib.w4_rms_add_q8(x, res, w, T, H, eps, h, out, qs, None)
    return lib.w4_rms_add(x, res, w, T, H, eps, h, out, None)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(H=0), BAD), (dict(H=12), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=1e31), BAD), (dict(H=32776), UNSUP), (dict(T=1 << 31), UNSUP), (dict(x=None), BAD), (dict(h=None), BAD),
    (dict(out=None), BAD), (dict(x=P + 2), BAD), (dict(res=P + 8), BAD), (dict(w=P + 2), BAD), (dict(h=P + 4), BAD),
    (dict(out=P + 4), BAD), (dict(T=0), _lib.W4_OK), (dict(T=0, x=None), _lib.W4_OK)])
def test_rms_add(q8, kw, want):
    assert rms(_lib.load(), q8, **kw) == want


def test_rms_add_q8_needs_scales():
    assert rms(_lib.load(), True, qs=None) == BAD
    assert rms(_lib.load(), True, qs=P + 2) == BAD


def lin(lib, xq=P, xs=P, codes=P, scales=P, y=P, M=4, N=64, K=256, ws=P, nws=1 << 40):
    return lib.w4a8_linear(xq, xs, codes, scales, y, M, N, K, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=48), BAD), (dict(N=(1 << 30) + 1), BAD),
    (dict(K=1 << 31), BAD), (dict(xq=None), BAD), (dict(xs=None), BAD), (dict(codes=None), BAD),
    (dict(scales=None), BAD), (dict(y=None), BAD), (dict(xq=P + 8), BAD), (dict(xs=P + 2), BAD),
    (dict(codes=P + 4), BAD), (dict(scales=P + 1), BAD), (dict(y=P + 2), BAD), (dict(ws=P + 8), BAD),
    (dict(M=1 << 30, N=1 << 20), UNSUP), (dict(M=0), _lib.W4_OK), (dict(M=0, xq=None, xs=None, y=None), _lib.W4_OK)])
def test_w4a8_linear(kw, want):
    assert lin(_lib.load(), **kw) == want


CACHE = dict(kind=_lib.W4_KV_INT8, heads=2, dim=64, pages=4, page=16, kc=P, vc=P, ks=P, vs=P)
BAD_CACHES = [
    (dict(kind=3), BAD), (dict(kind=-1), BAD), (dict(heads=0), BAD), (dict(dim=0), BAD), (dict(pages=0), BAD),
    (dict(page=0), BAD), (dict(kc=None), BAD), (dict(vc=None), BAD), (dict(ks=None), BAD), (dict(vs=None), BAD),
    (dict(kc=P + 8), BAD), (dict(vc=P + 4), BAD), (dict(ks=P + 1), BAD), (dict(pages=1 << 31), UNSUP)]


def write(lib, k=P, v=P, kst=128, vst=128, slots=P, T=5, **over):
    c = {**CACHE, **over}
    return lib.kv_cache_write(k, v, kst, vst, slots, T, c["kind"], c["heads"], c["dim"], c["pages"], c["page"],
                              c["kc"], c["vc"], c["ks"], c["vs"], None, None)


def read(lib, k=P, v=P, slots=P, T=5, **over):
    c = {**CACHE, **over}
    return lib.kv_cache_read(slots, T, c["kind"], c["heads"], c["dim"], c["pages"], c["page"], c["kc"], c["vc"],
                             c["ks"], c["vs"], k, v, None, None)


def attend(lib, q=P, qst=256, table=P, width=3, lens=P, B=2, q_heads=4, scale=0.1, softcap=0.0, window=0, out=P,
           lse=P, ws=P, nws=1 << 40, **over):
    c = {**CACHE, **over}
    return lib.kv_cache_attend(q, qst, c["kc"], c["vc"], c["ks"], c["vs"], c["kind"], table, width, lens, B, q_heads,
                               c["heads"], c["dim"], c["pages"], c["page"], scale, softcap, window, out, lse, ws, nws,
                               None, None)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_caches(call, kw, want):
    assert call(_lib.load(), **kw) == want


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(dim=48), BAD), (dict(dim=1056), UNSUP), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(slots=None), BAD), (dict(k=P + 8), BAD), (dict(slots=P + 4), BAD), (dict(T=0), _lib.W4_OK),
    (dict(T=0, k=None, v=None, slots=None), _lib.W4_OK)])
def test_rows(call, kw, want):
    assert call(_lib.load(), **kw) == want


@pytest.mark.parametrize("kw", [dict(kst=120), dict(vst=132), dict(kst=-128)])
def test_write_strides(kw):
    assert write(_lib.load(), **kw) == BAD


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), BAD), (dict(q_heads=3), BAD), (dict(q_heads=0), BAD), (dict(width=0), BAD), (dict(window=-1), BAD),
    (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(softcap=-1.0), BAD),
    (dict(softcap=float("nan")), BAD), (dict(dim=96, qst=384), UNSUP), (dict(dim=512, qst=2048), UNSUP),
    (dict(q_heads=65538, qst=1 << 40), UNSUP), (dict(width=1 << 30), UNSUP), (dict(qst=248), BAD), (dict(qst=260), BAD),
    (dict(q=None), BAD), (dict(table=None), BAD), (dict(lens=None), BAD), (dict(out=None), BAD), (dict(q=P + 8), BAD),
    (dict(out=P + 8), BAD), (dict(lse=P + 2), BAD), (dict(ws=P + 8), BAD), (dict(ks=P + 2), BAD), (dict(B=0), _lib.W4_OK)])
def test_attend(kw, want):
    assert attend(_lib.load(), **kw) == want


def test_workspaces_too_small():
    lib = _lib.load()
    for need, call in ((lib.w4_workspace_bytes(_lib.W4_OP_ATTEND, 2, 4, 64, 2, 0), attend),
                       (lib.w4_workspace_bytes(_lib.W4_OP_LINEAR_8, 4, 64, 256, 1, 1), lin)):
        if need:
            assert call(lib, nws=need - 1) == WS and call(lib, ws=None) == WS
    assert lib.w4_workspace_bytes(_lib.W4_OP_ATTEND, -1, 4, 64, 2, 0) == 0


def test_binding_refuses_what_is_not_on_a_device():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: api.w4_rms_add(x), lambda: api.w4_rms_add_q8(x),
                 lambda: api.w4a8_linear(x.to(torch.int8), x, x, x), lambda: api.kv_cache_write(x, x, x, x, x),
                 lambda: api.kv_cache_read(x, x, x), lambda: api.kv_cache_attend(x, x, x, x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        api.w4_rms_add([1.0])
    with pytest.raises(ValueError):
        api.KVCache(1, 1, 1, 64, "int2", device="cpu")
    with pytest.raises(ValueError):
        api.KVCache(1, 1, 1, 40, device="cpu")


def test_cache_slots_and_bytes():
    c = api.KVCache(6, 2, 16, 64, "int4", device="cpu")
    assert c.nbytes() == 2 * (6 * 2 * 16) * (64 // 2 + 2 * 2)
    table = torch.tensor([[4, 1], [0, -1], [2, 5]], dtype=torch.int32)
    assert c.slots(table, torch.tensor([17, 3, -1], dtype=torch.int32)).tolist() == [17, 3, -1]
    # a position on a page that is not there stays padded
    assert c.slots(table, torch.tensor([0, 16, 31])).tolist()[1] < 0
    assert c.slots(table, torch.tensor([0, 16, 31])).tolist()[::2] == [64, 95]
    words = torch.full((1,), -0x77777778, dtype=torch.int32)
    assert (c.k == words).all() and not c.k_scales.any()


def test_packed_calls():
    """w4_packed: the same answers as the entry points, and its own refusals."""
    import struct
    lib = _lib.load()

    def packed(entry, fmt, *values, words=None):
        return lib.w4_packed(entry, struct.pack("=q" + fmt, len(values) if words is None else words, *values))

    rms_fmt = "QQQqqdQQQ"
    good = (P, 0, 0, 0, 64, 1e-6, 0, P, 0)                       # no rows: nothing to do
    assert packed(_lib.W4_ENTRY_RMS_ADD, rms_fmt, *good) == _lib.W4_OK
    assert packed(_lib.W4_ENTRY_RMS_ADD, rms_fmt, *good, words=8) == BAD
    assert packed(99, rms_fmt, *good) == BAD and packed(0, rms_fmt, *good) == BAD
    assert lib.w4_packed(_lib.W4_ENTRY_RMS_ADD, None) == BAD
    # an integer past its parameter (H is 32 bits), and the entry point's own refusals
    assert packed(_lib.W4_ENTRY_RMS_ADD, rms_fmt, P, 0, 0, 0, (1 << 32) + 64, 1e-6, 0, P, 0) == BAD
    assert packed(_lib.W4_ENTRY_RMS_ADD, rms_fmt, P, 0, 0, 4, 12, 1e-6, 0, P, 0) == BAD
    assert packed(_lib.W4_ENTRY_RMS_ADD, rms_fmt, P, 0, 0, 4, 64, -1.0, 0, P, 0) == BAD
    assert packed(_lib.W4_ENTRY_RMS_ADD, rms_fmt, P, 0, 0, 4, 32776, 0.0, 0, P, 0) == UNSUP
    with pytest.raises(_lib.W4Error, match="kv_cache_read failed: W4_ERR_INVALID_ARG"):
        _lib.kv_read(P, 5, 7, 2, 64, 4, 16, P, P, P, P, P, P, 0, 0)
    _lib.kv_read(P, 0, _lib.W4_KV_INT8, 2, 64, 4, 16, P, P, P, P, P, P, 0, 0)
    with pytest.raises(_lib.W4Error):
        _lib.kv_attend(P, 256, P, P, P, P, 1, P, 3, P, 2, 4, 2, 64, 4, 16, float("nan"), 0.0, 0, P, 0, P, 1 << 20, 0, 0)


def test_first_tensor_by_its_name():
    """Every argument may be named, the first among them."""
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: api.w4_rms_add(x=x), lambda: api.w4_rms_add_q8(x=x),
                 lambda: api.w4a8_linear(xq=x, xs=x, codes=x, scales=x),
                 lambda: api.kv_cache_write(k=x, v=x, slots=x, k_cache=x, v_cache=x),
                 lambda: api.kv_cache_read(slots=x, k_cache=x, v_cache=x),
                 lambda: api.kv_cache_attend(q=x, k_cache=x, v_cache=x, page_table=x, seq_lens=x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="x: expected a torch.Tensor"):
        api.w4_rms_add()


def test_slots_of_positions_outside_the_table():
    cache = api.KVCache(4, 1, 16, 32, "int8", device="cpu")
    table = torch.tensor([[2, 0], [1, 3], [0, -1], [3, 9]], dtype=torch.int32)
    at = lambda *p: cache.slots(table, torch.tensor(p, dtype=torch.int32)).tolist()
    assert at(5, 16, -1, 0) == [37, 48, -1, 48]
    past = at(32, 1 << 30, 4096, 17)
    assert all(s >= 4 * 16 for s in past)                   # reported and dropped by a write
    with pytest.raises(ValueError):
        cache.slots(table[:, :0], torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        cache.slots(table, torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("eps,rows", [(None, 4), ("1", 4), (1e-6, 4.5), (1e-6, None), (1e-6, 1 << 70)])
def test_values_of_the_wrong_kind_are_type_errors(eps, rows):
    with pytest.raises(TypeError, match="w4_rms_add"):
        _lib.rms_add(P, 0, 0, rows, 64, eps, 0, P, 0)


@pytest.mark.parametrize("q,out", [(P, P), (P, P + 1008), (P + 1008, P), (P + 512, P)])
def test_attention_refuses_outputs_over_queries(q, out):
    assert attend(_lib.load(), q=q, out=out) == BAD           # (two rows of 4 heads of 64: 1024 bytes each)
