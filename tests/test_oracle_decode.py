"""Pins of oracle/decode.py by hand-worked values (CPU only)."""
import numpy as np

from oracle import bf16, decode, q4


def test_norm_of_a_hand_worked_row():
    x = bf16.from_f64(np.array([[3.0, -1.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]]))
    r = bf16.from_f64(np.array([[1.0, 1.0, 0.0, 0.0, 0.0, 0.0, 0.0, 2.0]]))
    h, y = decode.rms_add(x, r, None, 0.0)
    assert bf16.to_f64(h)[0].tolist() == [4, 0, 0, 0, 0, 0, 0, 2]
    assert np.allclose(y[0, 0], 4 / np.sqrt(20 / 8), rtol=1e-15)
    w = bf16.from_f64(np.full(8, 0.5))
    assert np.allclose(decode.rms_add(x, r, w, 0.0)[1], y / 2, rtol=1e-15)


def test_row_codes_of_hand_worked_groups():
    v = np.zeros((1, 64))
    v[0, 0], v[0, 1], v[0, 2] = 127.0, -127.0, 0.5          # step 1: 0.5 ties to 0
    v[0, 32] = np.inf
    q, s = decode.quantise_rows(bf16.from_f64(v), "int8")
    assert q[0, :4].tolist() == [127, -127, 0, 0]
    assert bf16.to_f64(s)[0, 0] == 1.0 and s[0, 1] == bf16.QNAN_BITS and not q[0, 32:].any()
    q, s = decode.quantise_rows(bf16.from_f64(v[:, :32] * 7 / 127), "int4")
    assert q[0, :2].tolist() == [7, -7]
    w = decode.pack_l1(q)
    assert (w[0, 0] & 0xFF) == 0x1F and (w[0, 1:4] == 0x88888888).all()
    one = np.full((1, 1), 0x3F80, np.uint16)
    assert (q4.dequant(w, one) == q).all()


def test_quotients_stay_clear_of_halves():
    """The codes do not depend on whether x / s is taken in float32 or float64: over every pair of
    8-bit significands the float32 quotient rounds to the same integer."""
    a = np.arange(128, 256, dtype=np.float64)
    for shift in range(0, 10):
        num, den = a[:, None], a[None, :] * 2.0 ** (shift - 7)
        exact, short = num / den, (num.astype(np.float32) / den.astype(np.float32)).astype(np.float64)
        assert (np.rint(exact) == np.rint(short)).all()


def test_attention_of_two_tokens():
    q = np.array([1.0, 0.0])
    k = np.array([[0.0, 5.0], [np.log(3.0), 0.0]])
    v = np.array([[4.0, 0.0], [0.0, 8.0]])
    out, lse, *_ = decode.attend(q, k, v, 1.0)
    assert np.allclose(out, [1.0, 6.0]) and np.isclose(lse, np.log(4.0))
    assert np.allclose(decode.attend(q, k, v, 1.0, window=1)[0], v[1])
    out, lse, *_ = decode.attend(q, k[:0], v[:0], 1.0)
    assert not out.any() and lse == -np.inf
    assert np.isclose(decode.attend(q, k, v, 1.0, softcap=0.5)[1],
                      np.log(1 + np.exp(0.5 * np.tanh(2 * np.log(3.0)))))


def test_linear_matches_group_by_group():
    r = np.random.RandomState(0)
    xq = r.randint(-127, 128, (3, 96)).astype(np.int8)
    q = r.randint(-8, 8, (5, 96))
    s = bf16.from_f64(r.rand(5, 3) + 0.1)
    xs = np.array([0.5, 1.0, 2.0], np.float32)
    y = decode.w4a8_linear(xq, xs, decode.pack_l1(q), s)
    want = np.zeros((3, 5))
    for m in range(3):
        for n in range(5):
            for g in range(3):
                want[m, n] += xs[m] * bf16.to_f64(s)[n, g] * int(
                    (xq[m, 32 * g:32 * g + 32].astype(int) * q[n, 32 * g:32 * g + 32]).sum())
    assert np.allclose(y, want, rtol=1e-13)
    assert (decode.w4a8_magnitude(xq, xs, decode.pack_l1(q), s) >= np.abs(want) - 1e-9).all()
