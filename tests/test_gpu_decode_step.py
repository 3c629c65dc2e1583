"""A decode step through attention blocks and expert layers, as a user runs it: the calls together, step
after step over a growing cache, eager and captured, on both expert paths, and beside the oracle
operator by operator on the step's own intermediate values (the operators' own tolerances)."""
import numpy as np
import pytest
import torch

from oracle import bf16, decode, linear
from w4a16_group_quantized_w4_b200 import api, stack
from tests._util import assert_rows_close, dev_bf16, dev_u32, host_bf16_bits, host_f64, host_u32

pytestmark = pytest.mark.gpu

L, E, K, H, I = 2, 16, 4, 256, 128
HQ, HKV, D, PAGE = 6, 2, 64, 16


def weights(r, rows, cols):
    q = r.randint(-8, 8, (rows, cols))
    s = bf16.from_f64((0.5 + r.rand(rows, cols // 32)) * 0.25 / np.sqrt(cols))
    return decode.pack_l1(q), s


def build(kind, seed=0, B=5, positions=70):
    r = np.random.RandomState(seed)
    st = stack.MoEStack(L, E, K, H, I)
    for codes, scales in ((st.gu_codes, st.gu_scales), (st.dn_codes, st.dn_scales)):
        c, s = weights(r, codes.shape[0] * codes.shape[1] * codes.shape[2], codes.shape[3] * 8)
        codes.copy_(dev_u32(c).view(codes.shape))
        scales.copy_(dev_bf16(s).view(scales.shape))
    per_seq = -(-positions // PAGE)
    blocks = []
    for _ in range(L):
        qkv, o = weights(r, (HQ + 2 * HKV) * D, H), weights(r, H, HQ * D)
        norms = [dev_bf16(bf16.from_f64(1 + 0.2 * r.randn(H))) for _ in range(2)]
        blocks.append(stack.AttentionBlock(dev_u32(qkv[0]), dev_bf16(qkv[1]), dev_u32(o[0]), dev_bf16(o[1]),
                                           api.KVCache(B * per_seq, HKV, PAGE, D, kind), HQ, *norms))
    table = torch.from_numpy(r.permutation(B * per_seq).reshape(B, per_seq).astype(np.int32)).cuda()
    return st, blocks, table, r


def inputs(r, B):
    return (dev_bf16(bf16.from_f64(r.randn(B, H))),
            [torch.from_numpy(r.randn(B, E).astype(np.float32)).cuda() for _ in range(L)])


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("fused", [False, True])
def test_steps_match_the_calls_and_the_oracle(kind, fused):
    B = 5
    st, blocks, table, r = build(kind)
    start = np.array([0, 3, 17, 40, 60])                      # the sequences have different ages
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for step in range(4):
        x0, logits = inputs(r, B)
        pos = torch.from_numpy(start).cuda() + step if step else torch.from_numpy(start).cuda()
        if step == 0:                                         # fill the older positions as a prompt would
            for l, b in enumerate(blocks):
                seqs = np.repeat(np.arange(B), start)
                at = np.concatenate([np.arange(n) for n in start])
                k, v = (bf16.from_f64(r.randn(len(at), HKV, D)) for _ in range(2))
                slots = table.cpu().numpy()[seqs, at // PAGE].astype(np.int64) * PAGE + at % PAGE
                b.cache.write(dev_bf16(k), dev_bf16(v), torch.from_numpy(slots).cuda())
        slots = blocks[0].cache.slots(table, pos)
        lens.copy_((pos + 1).int())
        before = [(b.cache.k.clone(), b.cache.v.clone()) for b in blocks]
        out, h_out = st.decode_step(x0, logits, blocks, table, lens, slots, fused=fused)
        out, h_out = out.clone(), h_out.clone()
        # the same step from the single calls (writing the same rows again leaves the cache as it is)
        y, h = x0, None
        for l, b in enumerate(blocks):
            x_in, h_in = y, h
            n, ns, h = api.w4_rms_add_q8(x_in, h_in, b.norm_in)
            rows = api.w4a8_linear(n, ns, *b.qkv)
            q, k, v = rows.view(B, -1, D).split((HQ, HKV, HKV), dim=1)
            b.cache.write(k, v, slots)
            a = b.cache.attend(q, table, lens)
            o = api.w4a16_linear(a.view(B, -1), *b.o)
            x, h2 = api.w4_rms_add(o, h, b.norm_out)
            if l == 0 and step == 3:
                check_block(b, x_in, h_in, h, n, ns, rows, q, a, o, x, h2, table, lens)
            y, h = st.layer(l, B, fused)(x, logits[l]).clone(), h2
        want, want_h = api.w4_rms_add(y, h)
        assert torch.equal(out, want) and torch.equal(h_out, want_h)
        # nothing but the new rows of the caches changed
        for b, (ck, cv) in zip(blocks, before):
            keep = torch.ones(ck.shape[0] * PAGE, dtype=torch.bool, device="cuda")
            keep[slots] = False
            for now, old in ((b.cache.k, ck), (b.cache.v, cv)):
                rows_now, rows_old = (t.transpose(1, 2).reshape(-1, *t.shape[1:2], t.shape[3]) for t in (now, old))
                assert torch.equal(rows_now[keep], rows_old[keep])
    assert np.isfinite(host_f64(out)).all()


def check_block(b, x, h_in, h, n, ns, rows, q, a, o, y, h2, table, lens):
    """Every operator of one block against the oracle on the operator's own inputs."""
    res = None if h_in is None else host_bf16_bits(h_in)
    h_ref, n_ref = decode.rms_add(host_bf16_bits(x), res, host_bf16_bits(b.norm_in), api.RMS_EPS)
    assert np.array_equal(host_bf16_bits(h), h_ref)
    nq, s = n.cpu().numpy(), ns.cpu().numpy()
    assert (np.abs(nq - n_ref / s[:, None]) <= 0.5 + 1e-2).all()
    lin = decode.w4a8_linear(nq, s, host_u32(b.qkv[0]), host_bf16_bits(b.qkv[1]))
    assert_rows_close(host_f64(rows), lin, rel_l2=2.0 ** -8, max_abs_frac=2.0 ** -8)
    slots = [b.cache.slots(table, torch.full((table.shape[0],), p, device="cuda")) for p in range(int(lens.max()))]
    got = [b.cache.read(s) for s in slots]
    keys, values = (np.stack([host_f64(g[i]) for g in got]) for i in (0, 1))       # [position, seq, head, D]
    out = host_f64(a)
    for i, ln in enumerate(lens.tolist()):
        for hd in range(HQ):
            g = hd // (HQ // HKV)
            ref, _, mag, peak, vsum = decode.attend(host_f64(q)[i, hd], keys[:ln, i, g], values[:ln, i, g], D ** -0.5)
            # rows read back are rounded to bf16 (2^-8 of each, which scores and values both carry)
            tol = np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -9 + 2.0 ** -8 + 2 * 2.0 ** -8 * peak * D ** -0.5) + vsum * 2.0 ** -31
            assert (np.abs(out[i, hd] - ref) <= tol).all()
    assert_rows_close(host_f64(o), linear.w4a16_linear(host_bf16_bits(a.reshape(len(out), -1)), host_u32(b.o[0]),
                                                       host_bf16_bits(b.o[1])))
    h2_ref, y_ref = decode.rms_add(host_bf16_bits(o), host_bf16_bits(h), host_bf16_bits(b.norm_out), api.RMS_EPS)
    assert np.array_equal(host_bf16_bits(h2), h2_ref)
    assert_rows_close(host_f64(y), y_ref, rel_l2=2.0 ** -8, max_abs_frac=2.0 ** -8)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_captured_steps_replay_over_a_growing_cache(kind):
    """One captured step, replayed with new inputs, lengths and slots, gives the eager step's bits."""
    B = 5
    sides = [build(kind, seed=3) for _ in range(2)]
    x0, logits = inputs(sides[0][3], B)
    x0 = x0.clone()
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    slots = sides[0][1][0].cache.slots(sides[0][2], lens - 1)
    st, blocks, table, _ = sides[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.decode_step(x0, logits, blocks, table, lens, slots)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, h = st.decode_step(x0, logits, blocks, table, lens, slots)
    r = np.random.RandomState(9)
    for step in range(40):                                    # across page borders
        nx, nl = inputs(r, B)
        x0.copy_(nx)
        for a, b in zip(logits, nl):
            a.copy_(b)
        lens.fill_(step + 1)
        lens[2] = max(1, step)                                # one sequence is a token behind
        slots.copy_(blocks[0].cache.slots(table, lens - 1))
        g.replay()
        st2, blocks2, table2, _ = sides[1]
        want, want_h = st2.decode_step(nx, nl, blocks2, table2, lens, blocks2[0].cache.slots(table2, lens - 1))
        assert torch.equal(out, want) and torch.equal(h, want_h), step
    for a, b in zip(blocks, sides[1][1]):
        assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v, b.cache.v)


def test_block_refuses_weights_of_the_wrong_shape():
    _, blocks, _, _ = build("int8")
    b = blocks[0]
    with pytest.raises(ValueError):
        stack.AttentionBlock(*b.qkv, *b.o, b.cache, HQ + 1)
    with pytest.raises(ValueError):
        stack.AttentionBlock(*b.qkv, b.qkv[0], b.qkv[1], b.cache, HQ)
    st, blocks, table, r = build("int8")
    x0, logits = inputs(r, 5)
    with pytest.raises(ValueError):
        st.decode_step(x0, logits, blocks[:1], table, None, None)


def test_step_on_another_stream():
    st, blocks, table, r = build("int8", seed=4)
    x0, logits = inputs(r, 5)
    lens = torch.ones(5, dtype=torch.int32, device="cuda")
    slots = blocks[0].cache.slots(table, lens - 1)
    want = st.decode_step(x0, logits, blocks, table, lens, slots)[0].clone()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    got = st.decode_step(x0, logits, blocks, table, lens, slots, stream=other)[0]
    other.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_padded_rows_leave_the_others_alone(kind):
    """Rows of length 0 without a slot: whatever they hold, the others' results and the caches stay the same."""
    outs = []
    for other in range(2):
        st, blocks, table, r = build(kind, seed=6)
        x0, logits = inputs(r, 5)
        lens = torch.tensor([1, 0, 1, 0, 1], dtype=torch.int32, device="cuda")
        for step in range(3):
            if other:
                x0[[1, 3]] = 100 * torch.randn((2, H), device="cuda").to(torch.bfloat16)
            slots = blocks[0].cache.slots(table, lens - 1)
            assert (slots[[1, 3]] == -1).all()
            n, h = st.decode_step(x0, logits, blocks, table, lens, slots)
            lens += (lens > 0).int()
        outs.append((n[::2], h[::2], [b.cache.k for b in blocks], [b.cache.v for b in blocks]))
    a, b = outs
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for i in (2, 3):
        assert all(torch.equal(p, q) for p, q in zip(a[i], b[i]))


def test_two_captured_blocks_replayed_side_by_side():
    """Attention blocks captured one after the other share no scratch: replayed at once they give the eager bits."""
    sides = []
    for seed in (7, 8):
        _, blocks, table, r = build("int8", seed=seed)
        x, h = (dev_bf16(bf16.from_f64(r.randn(5, H))) for _ in range(2))
        lens = torch.full((5,), 40, dtype=torch.int32, device="cuda")
        slots = blocks[0].cache.slots(table, lens - 1)
        want = [t.clone() for t in blocks[0](x, h, table, lens, slots)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = blocks[0](x, h, table, lens, slots)
        # a graph reads its inputs where they were: they are kept with it
        sides.append((g, got, want, torch.cuda.Stream(), (blocks, x, h, table, lens, slots)))
    for _ in range(30):
        for g, _, _, stream, _ in sides:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for _, got, want, *_ in sides:
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_step_on_another_stream_keeps_its_tensors_there():
    """A step given a stream allocates on it: tensors that it drops are not handed to the current stream
    while its kernels still use them."""
    st, blocks, table, r = build("int8", seed=4)
    x0, logits = inputs(r, 5)
    lens = torch.ones(5, dtype=torch.int32, device="cuda")
    slots = blocks[0].cache.slots(table, lens - 1)
    want = st.decode_step(x0, logits, blocks, table, lens, slots)[0].clone()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(10):
        got = st.decode_step(x0, logits, blocks, table, lens, slots, stream=other)[0]
        spoil = [torch.full((5, H), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert len(spoil) == 8 and torch.equal(got, want)
