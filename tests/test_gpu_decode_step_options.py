"""An attention block's scale and eps, and what a decode step reports, beside the single calls."""
import pytest
import torch

from oracle import bf16
from w4a16_group_quantized_w4_b200 import _lib, api, stack
from tests._util import dev_bf16
from tests.test_gpu_decode_step import D, H, HKV, HQ, build, inputs

pytestmark = pytest.mark.gpu


def test_scale_and_eps_reach_the_calls():
    _, blocks, table, r = build("int8", seed=12)
    b = blocks[0]
    x, h0 = (dev_bf16(bf16.from_f64(0.01 * r.randn(5, H))) for _ in range(2))
    lens = torch.full((5,), 40, dtype=torch.int32, device="cuda")
    b.cache.k.random_(-9, 9)
    b.cache.v.random_(-9, 9)
    b.cache.k_scales.fill_(0.1)
    b.cache.v_scales.fill_(0.1)
    slots = b.cache.slots(table, lens - 1)
    plain = [t.clone() for t in b(x, h0, table, lens, slots)]
    other = stack.AttentionBlock(*b.qkv, *b.o, b.cache, HQ, b.norm_in, b.norm_out, scale=0.7, eps=0.01)
    got = other(x, h0, table, lens, slots)
    n, ns, h = api.w4_rms_add_q8(x, h0, b.norm_in, eps=0.01)
    q, k, v = api.w4a8_linear(n, ns, *b.qkv).view(5, -1, D).split((HQ, HKV, HKV), dim=1)
    b.cache.write(k, v, slots)
    o = api.w4a16_linear(b.cache.attend(q, table, lens, scale=0.7).view(5, -1), *b.o)
    want = api.w4_rms_add(o, h, b.norm_out, eps=0.01)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert not torch.equal(got[0], plain[0])


def test_a_step_reports_slots_lengths_and_pages_out_of_range():
    st, blocks, table, r = build("int8", seed=13)
    x0, logits = inputs(r, 5)
    lens = torch.ones(5, dtype=torch.int32, device="cuda")
    slots = blocks[0].cache.slots(table, lens - 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in st.decode_step(x0, logits, blocks, table, lens, slots)]
    got = st.decode_step(x0, logits, blocks, table, lens, slots, dev_status=status, eps=api.RMS_EPS)
    assert status.item() == _lib.W4_OK and all(torch.equal(p, q) for p, q in zip(got, want))
    past = slots.clone()
    past[1] = 1 << 40
    long_ = lens.clone()
    long_[3] = 1 << 20
    pages = table.clone()
    pages[2, 0] = 1 << 30
    for case in ((table, lens, past), (table, long_, slots), (pages, lens, slots)):
        status.zero_()
        st.decode_step(x0, logits, blocks, *case, dev_status=status)
        assert status.item() == _lib.W4_ERR_INVALID_ARG
