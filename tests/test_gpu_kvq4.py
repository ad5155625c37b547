"""GPU parity of the 4-bit KV cache (mlora_kv_write_q4, mlora_kv_read_q4) with
the oracle (oracle.kvq4).  Codes and scales follow from the inputs by fp32
divisions and roundings to nearest even, so they must match bit for bit, as
must every byte that a pass leaves alone; the read-back is one rounding to bf16
of an exact product and matches bit for bit too."""
import numpy as np
import pytest
import torch

from oracle import kvq4 as Q
from tests.gpu_util import dev, needs_gpu

pytestmark = pytest.mark.gpu


def _setup(g, B, H, D, bs, mb, unalloc=0.0):
    nb = B * mb + 3
    bt = g.permutation(nb)[:B * mb].reshape(B, mb).astype(np.int32)
    if unalloc:
        bt[g.random(bt.shape) < unalloc] = -1
    return bt, [g.integers(0, 256, (nb, H, bs, w), dtype=np.uint8) for w in (D // 2, D // 16, D // 2, D // 16)]


def _rows(g, shape, wide=True):
    v = g.standard_normal(shape) * (np.exp2(g.integers(-12, 9, shape[:1] + (1,))) if wide else 1.0)
    return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)


def _bits(t):
    return t.view(torch.int16).cpu().numpy()


def _check(ml, y, k_col, v_col, H, D, bt, seq, T, t0, cache, ku=1.0, vu=1.0, y_dev=None):
    want, st = Q.kv_write_q4(y.float().numpy(), k_col, v_col, H, D, bt, seq, T, t0, cache, ku, vu)
    ws = ml.Workspace(ml.kv_workspace_bytes())
    got = [dev(c) for c in cache]
    ml.kv_write_q4(y.cuda() if y_dev is None else y_dev, k_col, v_col, H, D, dev(bt), dev(seq), T, t0, *got, k_unit=ku,
                   v_unit=vu, ws=ws)
    assert ws.status() == st
    for i, (a, b) in enumerate(zip(got, want)):
        a = a.cpu().numpy()
        if i % 2 == 0:                               # codes of a NaN group stand for nothing
            nan = np.repeat(((want[i + 1] & 0x7F) == 0x7F), 8, -1)
            assert np.array_equal(np.where(nan, 0, a), np.where(nan, 0, b))
        else:
            assert np.array_equal(a, b)
    return got, want


@pytest.mark.parametrize("B,T,H,D,bs", [(1, 1, 8, 128, 16), (128, 5, 8, 128, 16), (7, 3, 2, 64, 1), (5, 17, 3, 48, 33),
                                        (3, 100, 1, 16, 20), (4, 9, 4, 256, 128)])
def test_write_bit_exact(B, T, H, D, bs):
    ml = needs_gpu()
    g = np.random.default_rng(B * T + D)
    mb = (T + 60) // bs + 2
    bt, cache = _setup(g, B, H, D, bs, mb)
    seq = g.integers(-3, mb * bs - T + 1, B).astype(np.int32)
    y = _rows(g, (B * T, 3 * H * D))
    _check(ml, y, H * D, 2 * H * D, H, D, bt, seq, T, 0, cache)


def test_every_bf16_ratio_to_the_scale():
    """Every finite bf16 magnitude against a group maximum that fixes the scale:
    all ties, the subnormal codes and the saturating ones."""
    ml = needs_gpu()
    H, D, bs = 1, 128, 16
    bits = np.arange(0, 0x7F80, dtype=np.uint32)
    for amax in (6.0, 5.5, 1.0, 0.0117, 2688.0, 3000.0, 1e-30):
        v = (bits << 16).view(np.float32)
        v = v[v <= amax][-15 * 8 * 400:]
        v = np.resize(v, (len(v) + 14) // 15 * 15).reshape(-1, 15)
        v = np.concatenate((v * np.where(np.arange(15) % 2, -1, 1), np.full((len(v), 1), amax)), 1)
        v = np.resize(v, ((len(v) + 7) // 8 * 8, 16)).reshape(-1, D).astype(np.float32)
        M = len(v)
        y = torch.from_numpy(np.concatenate((v, -v), 1)).to(torch.bfloat16)
        bt = np.arange((M + bs - 1) // bs, dtype=np.int32)[None]
        cache = [np.zeros((bt.shape[1], H, bs, w), np.uint8) for w in (64, 8, 64, 8)]
        _check(ml, y, 0, D, H, D, bt, np.zeros(1, np.int32), M, 0, cache)


def test_zeros_infinities_and_nan():
    ml = needs_gpu()
    g = np.random.default_rng(3)
    B, T, H, D, bs = 2, 4, 2, 64, 16
    bt, cache = _setup(g, B, H, D, bs, 2)
    y = _rows(g, (B * T, 2 * H * D), wide=False)
    y[0] = 0
    y[1] = -0.0
    y[2, 5] = float("nan")
    y[2, 200] = -float("nan")
    y[3, 40] = float("inf")
    y[4, 41] = -float("inf")
    y[5, :16] = 1e-41                                # bf16 subnormals
    y[6] = 3e38
    _check(ml, y, 0, H * D, H, D, bt, np.array([0, 9], np.int32), T, 0, cache)


@pytest.mark.parametrize("ku,vu", [(0.37, 5.5), (2.0 ** -20, 2.0 ** 20), (1e-30, 1e30)])
def test_units(ku, vu):
    ml = needs_gpu()
    g = np.random.default_rng(4)
    B, T, H, D, bs = 3, 7, 2, 128, 16
    bt, cache = _setup(g, B, H, D, bs, 3)
    y = _rows(g, (B * T, 2 * H * D))
    y[:, H * D:] *= vu
    y[:, :H * D] *= ku
    got, want = _check(ml, y, 0, H * D, H, D, bt, np.array([0, 9, 30], np.int32), T, 0, cache, ku, vu)
    _read_check(ml, got, want, bt, np.array([0, 9, 30]), np.array([7, 16, 37]), 7, ku, vu)


def _read_check(ml, got, cache, bt, start, end, rows, ku=1.0, vu=1.0):
    k, v, st = Q.kv_read_q4(cache, bt, start, end, rows, ku, vu)
    ws = ml.Workspace(ml.kv_workspace_bytes())
    kd, vd = ml.kv_read_q4(*got, dev(bt), dev(start.astype(np.int32)), dev(end.astype(np.int32)), rows, k_unit=ku,
                           v_unit=vu, ws=ws)
    assert ws.status() == st
    for a, b in ((kd, k), (vd, v)):
        # code * scale is exact and the product with the unit one fp32 rounding, on both sides
        w = torch.from_numpy(b.astype(np.float32)).to(torch.bfloat16)
        nan = torch.isnan(w)
        assert torch.equal(torch.isnan(a.cpu()), nan)
        assert np.array_equal(np.where(nan, 0, _bits(a)), np.where(nan, 0, _bits(w)))


@pytest.mark.parametrize("B,rows,H,D,bs", [(1, 1, 8, 128, 16), (9, 33, 2, 64, 20), (3, 70, 3, 48, 16), (2, 300, 1, 128, 1)])
def test_read_back(B, rows, H, D, bs):
    """Ragged ranges, ranges that end before they start, unused requests, bad pages, any scale byte."""
    ml = needs_gpu()
    g = np.random.default_rng(rows)
    mb = (rows + 20) // bs + 1
    bt, cache = _setup(g, B, H, D, bs, mb, unalloc=0.1 if B > 1 else 0.0)
    start = g.integers(0, 20, B)
    end = start + g.integers(-2, rows + 3, B)
    if B > 1:
        start[1] = -4
    _read_check(ml, [dev(c) for c in cache], cache, bt, start, end, rows)
    _read_check(ml, [dev(c) for c in cache], cache, bt, start, np.full(B, 2 ** 31 - 1), rows)  # past the table


def test_write_status_and_untouched_bytes():
    """Rows past the table, unallocated pages, unused requests: skipped, with the status bit of the bf16 cache."""
    ml = needs_gpu()
    g = np.random.default_rng(6)
    B, T, H, D, bs, mb = 6, 5, 2, 64, 16, 2
    bt, cache = _setup(g, B, H, D, bs, mb)
    bt[0, 0] = -1
    bt[1, 1] = 10 ** 6
    y = _rows(g, (B * T, 2 * H * D))
    for seq in ([0, 14, -1, 30, 2 ** 31 - 1, 3], [-1] * 6, [4, 5, -9, 20, 0, 3]):
        _check(ml, y, 0, H * D, H, D, bt, np.array(seq, np.int32), T, 0, cache)


def test_unaligned_rows_and_draft_steps():
    ml = needs_gpu()
    g = np.random.default_rng(7)
    B, H, D, bs = 5, 2, 64, 16
    bt, cache = _setup(g, B, H, D, bs, 3)
    seq = np.array([0, 15, 16, 30, 40], np.int32)
    for cols, ld in (((3, 3 + H * D), 300), ((0, H * D), 257), ((8, 8 + H * D), 272)):
        for t0 in (0, 2):
            _check(ml, _rows(g, (B, ld)), *cols, H, D, bt, seq, 1, t0, cache)
    y = _rows(g, (B, 2 * H * D))
    buf = torch.empty(y.numel() + 1, dtype=torch.bfloat16, device="cuda")
    view = buf[1:].view_as(y)
    view.copy_(y)
    _check(ml, y, 0, H * D, H, D, bt, seq, 1, 0, cache, y_dev=view)


def test_on_a_stream_and_in_a_graph():
    ml = needs_gpu()
    g = np.random.default_rng(8)
    B, T, H, D, bs = 4, 3, 2, 128, 16
    bt, cache = _setup(g, B, H, D, bs, 3)
    seq = np.array([0, 20, 5, 40], np.int32)
    y = _rows(g, (B * T, 2 * H * D))
    want, _ = Q.kv_write_q4(y.float().numpy(), 0, H * D, H, D, bt, seq, T, 0, cache)
    ws = ml.Workspace(ml.kv_workspace_bytes())
    got, yd, btd, sd = [dev(c) for c in cache], y.cuda(), dev(bt), dev(seq)
    end = sd + T
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ml.kv_write_q4(yd, 0, H * D, H, D, btd, sd, T, 0, *got, ws=ws)
        k, v = ml.kv_read_q4(*got, btd, sd, end, T, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gr.replay()
    s.synchronize()
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    rk, rv, _ = Q.kv_read_q4(want, bt, seq, seq + T, T)
    assert np.array_equal(k.double().cpu().numpy(), rk) and np.array_equal(v.double().cpu().numpy(), rv)
