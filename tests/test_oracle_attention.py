"""Pins for the oracles of attention over the paged cache and of the 4-bit
cache: cases worked by hand, closed forms and brute force."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle import kvq4 as Q


def test_e2m1_rounding_by_hand():
    v = [0, .2, .25, .26, .5, .74, .75, 1, 1.25, 1.26, 1.75, 2, 2.5, 2.51, 3.5, 4.9, 5, 5.1, 6, 7, 1e9, np.inf]
    want = [0, 0, 0, .5, .5, .5, 1, 1, 1, 1.5, 2, 2, 2, 3, 4, 4, 4, 6, 6, 6, 6, 6]
    assert Q.e2m1_decode(Q.e2m1_round(np.array(v))).tolist() == want
    assert Q.e2m1_decode(Q.e2m1_round(-np.array(v))).tolist() == [-x for x in want]
    assert Q.e2m1_decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_quantize_by_hand():
    # amax 12 -> scale 2; 1.0 / 2 = .5, 2.5 / 2 = 1.25 -> tie to 1, -12 / 2 = -6
    v = np.zeros(32, np.float32)
    v[0], v[1], v[5], v[15] = 1.0, 2.5, -12.0, 0.49
    codes, scales = Q.quantize(v)
    assert scales[0] == 0x40 and scales[1] == 0       # E4M3 of 2.0 and of 0
    assert codes.shape == (16,) and codes[0] == 1 | (2 << 4) and codes[2] == (15 << 4)
    d = Q.dequantize(codes, scales)
    assert d[:6].tolist() == [1.0, 2.0, 0, 0, 0, -12.0] and d[15] == 0.0 and not d[16:].any()
    # a unit moves the scale only
    c2, s2 = Q.quantize(v * 4, 4.0)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
    # a NaN takes its group and no other
    v[3] = np.nan
    v[20] = 1.0
    d = Q.dequantize(*Q.quantize(v))
    assert np.isnan(d[:16]).all() and d[20] == 1.03125   # 1/6 -> E4M3 0.171875; 5.82 -> 6


def test_quantize_error_bound():
    """|v - value| is at most half the largest step (1) of E2M1 times the scale,
    plus what saturation adds: the scale may round down by 1/16."""
    g = np.random.default_rng(0)
    v = (g.standard_normal((200, 64)) * np.exp(g.standard_normal((200, 1)))).astype(np.float32)
    codes, scales = Q.quantize(v)
    amax = np.abs(v).reshape(200, 4, 16).max(-1)
    err = np.abs(Q.dequantize(codes, scales) - v).reshape(200, 4, 16).max(-1)
    assert np.all(err <= amax / 6 * (1 + 1 / 16) + 2.0 ** -9)


def test_visible_by_brute_force():
    for pos in range(12):
        for w in range(0, 14):
            for s in range(0, 14):
                want = [j for j in range(pos + 1) if w == 0 or j > pos - w or j < s]
                assert OA.visible(pos, w, s).tolist() == want


def _dense(B, n, H, D, seed):
    g = np.random.default_rng(seed)
    k, v = g.standard_normal((2, B * n, 1, H, D))
    bt = np.arange(B * n, dtype=np.int32).reshape(B, n)
    return k, v, bt, (lambda page, off, h: (k[page, off, h], v[page, off, h]))


def test_closed_forms():
    B, n, H, D = 2, 9, 2, 16
    k, v, bt, of = _dense(B, n, H, D, 1)
    seq = np.array([5, 8], np.int32)
    # q = 0: the mean of the values seen
    o, st, _ = OA.attention(np.zeros((2, 4, D)), of, B, 1, 4, H, D, bt, 1, B * n, seq, 0, 0.3)
    assert st == 0
    for b in range(2):
        for hq in range(4):
            np.testing.assert_allclose(o[b, hq], v[b * n:b * n + seq[b] + 1, 0, hq // 2].mean(0), rtol=1e-12)
    # a window of one position sees its own value alone, whatever q
    o, _, _ = OA.attention(np.full((2, 4, D), 3.0), of, B, 1, 4, H, D, bt, 1, B * n, seq, 0, 0.3, window=1)
    for b in range(2):
        np.testing.assert_allclose(o[b, 3], v[b * n + seq[b], 0, 1], rtol=1e-12)
    # a very large score picks its position
    q = np.zeros((2, 4, D))
    q[0, 0] = 1e4 * k[3, 0, 0]
    sc = k[:6, 0, 0] @ q[0, 0]
    o, _, _ = OA.attention(q, of, B, 1, 4, H, D, bt, 1, B * n, seq, 0, 1.0)
    np.testing.assert_allclose(o[0, 0], v[int(sc.argmax()), 0, 0], rtol=1e-12)


def test_empty_rows_and_bad_slots():
    B, n, H, D = 3, 4, 1, 16
    k, v, bt, of = _dense(B, n, H, D, 2)
    bt[1] = -1
    bt[2, 2] = 99
    seq = np.array([-1, 2, 3], np.int32)
    o, st, _ = OA.attention(np.ones((3, 2, D)), of, B, 1, 2, H, D, bt, 1, B * n, seq, 0, 0.25)
    assert st == OA.BAD_SLOT and not o[0].any() and not o[1].any()
    z = 0.25 * k[8:12, 0, 0].sum(-1)
    p = np.exp(z) * np.array([1, 1, 0, 1])
    np.testing.assert_allclose(o[2, 0], p @ v[8:12, 0, 0] / p.sum(), rtol=1e-12)


def test_rows_of_a_pass_are_causal():
    """Row t of a verify pass equals a single row at its own position."""
    B, n, H, D = 2, 12, 2, 16
    _, _, bt, of = _dense(B, n, H, D, 3)
    q = np.random.default_rng(4).standard_normal((2 * 4, 4, D))
    seq = np.array([3, 7], np.int32)
    o, _, _ = OA.attention(q, of, B, 4, 4, H, D, bt, 1, B * n, seq, 0, 0.3, window=3, sinks=2)
    for t in range(4):
        o1, _, _ = OA.attention(q[t::4], of, B, 1, 4, H, D, bt, 1, B * n, seq, t, 0.3, window=3, sinks=2)
        np.testing.assert_allclose(o[t::4], o1, rtol=1e-13)


@pytest.mark.parametrize("unit", [1.0, 0.3])
def test_write_then_read_back(unit):
    g = np.random.default_rng(5)
    B, H, D, bs, mb, T = 3, 2, 32, 4, 4, 5
    nb = B * mb + 1
    bt = g.permutation(nb)[:B * mb].reshape(B, mb).astype(np.int32)
    cache = [np.full((nb, H, bs, w), 0x5A, np.uint8) for w in (D // 2, D // 16, D // 2, D // 16)]
    y = g.standard_normal((B * T, 3 * H * D)).astype(np.float32)
    seq = np.array([0, 7, -1], np.int32)
    new, st = Q.kv_write_q4(y, H * D, 2 * H * D, H, D, bt, seq, T, 0, cache, unit, unit)
    assert st == 0
    k, v, st = Q.kv_read_q4(new, bt, seq, seq + T, T + 2, unit, unit)
    assert st == 0 and not k[2].any() and not v[:, T:].any()
    for b in range(2):
        for t in range(T):
            c, s = Q.quantize(y[b * T + t, H * D:2 * H * D].reshape(H, D), unit)
            assert np.array_equal(k[b, t], Q.dequantize(c, s, unit))
    changed = sum(int((new[0][i] != cache[0][i]).any(-1).sum()) for i in range(nb))
    assert changed <= 2 * T * H
    _, st = Q.kv_write_q4(y, H * D, 2 * H * D, H, D, bt, np.array([13, 0, -1]), T, 0, cache)
    assert st == Q.BAD_SLOT
