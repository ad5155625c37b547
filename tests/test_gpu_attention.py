"""GPU parity of attention over the paged cache (mlora_attention,
mlora_attention_q4) with the float64 oracle (oracle.attention).

Tolerance per output entry, from the roundings the call makes (u(t) is half a
step of type t relative to the value: bf16 2^-8, fp16 2^-11, fp32 2^-24):
  * the output's own rounding: u(bf16) |o|;
  * the weights p enter the second product rounded: u(bf16) A over the bf16
    cache and u(fp16) A over the 4-bit one (A = sum p |v|, what a relative
    change of every weight can move), with fp16's subnormal half step 2^-25 on
    each of n weights, relative to a sum of weights that is at least 1:
    n 2^-25 max|v|;
  * a score is a fp32 sum of D products (and its scaling): at most (D + 4)
    u(fp32) S off, S = scale sum |q k|; over the 4-bit cache q is held in fp16
    relative to its row's largest entry, half a step 2^-25 of it at worst:
    D 2^-25 scale max|q| max|k| more.  A score off by d changes a weight by the
    factor e^d and the normalisation by another: 2 d A for small d;
  * exponentials (2^-22 each) and fp32 sums of n terms, above and below:
    2 (n + 8) u(fp32) A.
"""
import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import kvq4 as Q
from tests.gpu_util import dev, needs_gpu

pytestmark = pytest.mark.gpu

BAD_SLOT = 1 << 7


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _tolerance(o, bound, D, q4):
    A, S, n = bound["A"], bound["S"][..., None], bound["n"][..., None]
    d = (D + 4) * 2.0 ** -24 * S
    t = 2.0 ** -8 * np.abs(o) + 2 * (n + 8) * 2.0 ** -24 * A + 8 * 2.0 ** -22 * A
    if q4:
        d = d + D * 2.0 ** -25 * bound["qk"][..., None]
        t = t + 2.0 ** -11 * A + n * 2.0 ** -25 * bound["v"]
    else:
        t = t + 2.0 ** -8 * A
    return t + 2 * d * A + 1e-30


class Case:
    """A cache filled with random values, a table, and a pass's rows."""

    def __init__(self, q4, lens, T, Hq, H, D, bs, seed=0, t0=0, spread=1.0, pad=0, extra=3, unit=(1.0, 1.0)):
        g = np.random.default_rng(seed)
        self.q4, self.T, self.Hq, self.H, self.D, self.bs, self.t0 = q4, T, Hq, H, D, bs, t0
        self.seq = np.array(lens, np.int32)
        B = len(lens)
        mb = max(1, max((max(L, 0) + t0 + T + bs - 1) // bs for L in lens))
        nb = B * mb + extra
        self.bt = g.permutation(nb)[:B * mb].reshape(B, mb).astype(np.int32)
        self.y = _bf16(g.standard_normal((B * T, Hq * D + pad)) * spread)
        self.k = _bf16(g.standard_normal((nb, bs, H, D)) * np.exp(0.5 * g.standard_normal(D)))
        self.v = _bf16(g.standard_normal((nb, bs, H, D)))
        self.unit = unit
        if q4:
            self.quantize()

    def quantize(self):
        f = lambda t: t.float().numpy().transpose(0, 2, 1, 3)  # noqa: E731
        self.cache = [*Q.quantize(f(self.k), self.unit[0]), *Q.quantize(f(self.v), self.unit[1])]

    def keys(self):
        if not self.q4:
            k, v = self.k.double().numpy(), self.v.double().numpy()
            return lambda page, off, h: (k[page, off, h], v[page, off, h])
        k = Q.dequantize(self.cache[0], self.cache[1], self.unit[0])
        v = Q.dequantize(self.cache[2], self.cache[3], self.unit[1])
        return lambda page, off, h: (k[page, h, off], v[page, h, off])

    def oracle(self, scale=None, window=0, sinks=0, q_col=0):
        D = self.D
        q = self.y.double().numpy()[:, q_col:q_col + self.Hq * D].reshape(-1, self.Hq, D)
        nb = self.k.shape[0]
        return OA.attention(q, self.keys(), len(self.seq), self.T, self.Hq, self.H, D, self.bt, self.bs, nb, self.seq,
                            self.t0, D ** -0.5 if scale is None else scale, window, sinks)

    def device(self):
        self.y_d, self.bt_d, self.seq_d = self.y.cuda(), dev(self.bt), dev(self.seq)
        self.c_d = [dev(c) for c in self.cache] if self.q4 else [self.k.cuda(), self.v.cuda()]
        return self

    def call(self, ml, scale=None, window=0, sinks=0, q_col=0, y=None, **kw):
        y = self.y_d if y is None else y
        fn = ml.attention_q4 if self.q4 else ml.attention
        if self.q4:
            kw.update(k_unit=self.unit[0], v_unit=self.unit[1])
        return fn(y, q_col, self.Hq, *self.c_d, self.bt_d, self.seq_d, self.T, self.t0, scale=scale, window=window,
                  sinks=sinks, **kw)

    def check(self, ml, status=0, **kw):
        ws = ml.Workspace(ml.attention_workspace_bytes(len(self.seq) * self.T, self.T, self.Hq, self.H, self.D))
        out = self.device().call(ml, ws=ws, **kw)
        got = out.double().cpu().numpy().reshape(-1, self.Hq, self.D)
        o, st, bound = self.oracle(**kw)
        assert st == status and ws.status() == status
        tol = _tolerance(o, bound, self.D, self.q4)
        with np.errstate(invalid="ignore"):
            bad = ~(np.abs(got - o) <= tol) & ~(np.isnan(got) & np.isnan(o)) & ~(got == o)   # equal infinities
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                               float(np.nanmax(np.abs(got - o) / tol)))
        return out, o


both = pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])


@both
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8])
def test_draft_rows(q4, D, G):
    """One row a request; committed lengths around every tile size."""
    ml = needs_gpu()
    lens = [0, 1, 7, 14, 15, 16, 30, 31, 32, 33, 62, 63, 64, 65, 126, 127, 128, 129, 300, 511, 777]
    Case(q4, lens, 1, 2 * G, 2, D, 16, seed=G).check(ml)


@both
@pytest.mark.parametrize("T,G,D", [(2, 4, 128), (3, 5, 128), (5, 5, 128), (5, 4, 64), (9, 4, 128), (17, 7, 64), (17, 7, 128),
                                   (33, 2, 128), (17, 1, 128)])
def test_verify_rows(q4, T, G, D):
    """k + 1 rows a request, each blind to the rows after it."""
    ml = needs_gpu()
    Case(q4, [0, 3, 27, 31, 32, 60, 123, 128, 250, 400], T, 2 * G, 2, D, 16, seed=T).check(ml)


@both
@pytest.mark.parametrize("T,lens,Hq,H,D", [(130, [0, 5], 4, 2, 128), (257, [64], 4, 1, 64), (300, [200, 0], 3, 3, 128),
                                           (129, [127, 1, 300], 5, 1, 128), (64, [0, 640], 8, 1, 64)])
def test_prompt_rows(q4, T, lens, Hq, H, D):
    """Rows of a prompt or a piece of one."""
    ml = needs_gpu()
    c = Case(q4, lens, T, Hq, H, D, 32, seed=T)
    c.check(ml)
    c.check(ml, window=100, sinks=5)


@both
@pytest.mark.parametrize("bs", [1, 3, 16, 20, 33, 64, 128, 200])
def test_page_sizes(q4, bs):
    """Pages of any size: powers of two or not, ending inside a tile or past it."""
    ml = needs_gpu()
    Case(q4, [0, 5, 63, 64, 199, 333], 3, 8, 2, 128, bs, seed=bs).check(ml)


@both
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (31, 4), (32, 4), (33, 4), (100, 0), (100, 16),
                                          (128, 200), (1000, 4), (0, 7), (5, 100000)])
@pytest.mark.parametrize("T,D", [(1, 128), (5, 64)])
def test_window_and_sinks(q4, window, sinks, T, D):
    """Windows of one position, around the tile sizes and longer than the
    context; sinks inside, beside and beyond the window."""
    ml = needs_gpu()
    Case(q4, [0, 1, 4, 31, 32, 33, 64, 99, 131, 257, 640], T, 8, 2, D, 16, seed=window + sinks).check(
        ml, window=window, sinks=sinks)


@both
@pytest.mark.parametrize("D,Hq,H", [(16, 2, 1), (48, 6, 2), (80, 5, 5), (96, 8, 1), (192, 4, 2), (256, 4, 4)])
def test_other_head_sizes(q4, D, Hq, H):
    ml = needs_gpu()
    c = Case(q4, [0, 5, 40, 100], 3, Hq, H, D, 16, seed=D)
    c.check(ml)
    c.check(ml, window=9, sinks=2)


@both
def test_long_contexts_split_over_the_gpu(q4):
    """Few rows over long contexts: the positions are split over many CTAs and joined."""
    ml = needs_gpu()
    c = Case(q4, [5000, 1, 20001], 1, 8, 2, 128, 64, seed=1, spread=3.0)
    c.check(ml)
    c.check(ml, window=7000, sinks=64)
    Case(q4, [9999], 5, 5, 1, 128, 16, seed=2).check(ml)


@both
def test_many_requests_of_mixed_lengths(q4):
    ml = needs_gpu()
    g = np.random.default_rng(0)
    lens = np.where(g.random(200) < 0.1, -1, np.exp(g.uniform(0, 6.5, 200)).astype(np.int64))
    Case(q4, lens.tolist(), 2, 4, 2, 64, 16, seed=3).check(ml)


@both
def test_scores_of_large_range(q4):
    """Scores that spread over hundreds: the running maximum moves late and far."""
    ml = needs_gpu()
    c = Case(q4, [700, 64, 2000], 3, 8, 2, 128, 16, seed=5, spread=20.0)
    c.check(ml)
    # scores that rise along the context
    c = Case(q4, [1500], 2, 4, 1, 64, 16, seed=6)
    c.y = _bf16(np.ones((2, 4 * 64)))
    ramp = np.zeros((c.k.shape[0], 16, 1, 64), np.float32)
    for j in range(1502):
        ramp[c.bt[0, j // 16], j % 16] = 0.02 * j
    c.k = _bf16(ramp)
    if q4:
        c.quantize()
    c.check(ml)
    c.check(ml, scale=-0.125)     # and fall


@both
def test_scale_zero_is_the_mean(q4):
    ml = needs_gpu()
    Case(q4, [100, 40], 2, 4, 2, 128, 16).check(ml, scale=0.0)


@both
def test_unused_requests_and_empty_rows(q4):
    """Unused request slots and rows whose every page lies outside the cache are zeros."""
    ml = needs_gpu()
    for D in (64, 128, 80):
        c = Case(q4, [-1, 50, 20, -7, 300], 5, 8, 2, D, 16, seed=D)
        c.bt[2] = -1
        out, o = c.check(ml, status=BAD_SLOT)
        got = out.float().cpu().numpy().reshape(5, 5, -1)
        assert not got[0].any() and not got[2].any() and not got[3].any() and got[1].any()


@both
@pytest.mark.parametrize("T", [1, 5, 70])
def test_bad_pages_and_positions_past_the_table(q4, T):
    """Pages outside the cache and positions past the table are not seen; the others are."""
    ml = needs_gpu()
    c = Case(q4, [100, 200, 60], T, 8, 2, 128, 16, seed=9)
    c.bt[0, 3] = -5
    c.bt[1, 0] = c.k.shape[0]
    c.bt[1, 8] = 2 ** 31 - 1
    c.check(ml, status=BAD_SLOT)
    c.check(ml, status=BAD_SLOT, window=150, sinks=4)
    c = Case(q4, [100, 40], T, 8, 2, 128, 16, seed=10)
    c.bt = np.ascontiguousarray(c.bt[:, :4])       # 64 positions; request 0's rows lie past them
    c.check(ml, status=BAD_SLOT)
    c.check(ml, status=BAD_SLOT, window=60, sinks=4)
    # a length at the end of int32, its window wholly past the table
    c.seq[0] = -1
    o, _, bound = c.oracle(window=1000)
    c.seq[0] = 2 ** 31 - 1
    ws = ml.Workspace(ml.attention_workspace_bytes(2 * T, T, 8, 2, 128))
    got = c.device().call(ml, window=1000, ws=ws).double().cpu().numpy().reshape(o.shape)
    assert ws.status() == BAD_SLOT and not got[:T].any()
    assert np.all(np.abs(got - o) <= _tolerance(o, bound, 128, q4))


@both
@pytest.mark.parametrize("D", [64, 128, 48])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_nan_and_infinities_in_hidden_places(q4, D, T):
    """What no row sees, and what only later rows see, leaves a row alone."""
    ml = needs_gpu()
    for window, sinks in ((0, 0), (20, 3)):
        c = Case(q4, [0, 37, 90], T, 8, 2, D, 16, seed=11)
        k, v = (c.cache[1], c.cache[3]) if q4 else (c.k, c.v)
        at = (lambda blk, off: (blk, slice(None), off)) if q4 else (lambda blk, off: (blk, off))
        poison = (0x7F, 0x7F) if q4 else (float("inf"), float("nan"))
        used = set()
        for b in range(3):
            for j in range(int(c.seq[b]) + T):
                used.add((int(c.bt[b, j // 16]), j % 16))
            if window and c.seq[b] >= 30:
                used -= {(int(c.bt[b, j // 16]), j % 16) for j in range(5, int(c.seq[b]) - window)}
        for blk in range(c.k.shape[0]):
            for off in range(16):
                if (blk, off) not in used:
                    k[at(blk, off)] = poison[0]
                    v[at(blk, off)] = poison[1]
        if T > 1:                                    # request 1's last rows hold poison that they themselves see
            for j in (37 + T - 2, 37 + T - 1):
                v[at(int(c.bt[1, j // 16]), j % 16)] = poison[1]
        out, o = c.check(ml, window=window, sinks=sinks)
        got = out.float().cpu().numpy().reshape(3, T, -1)
        assert np.isfinite(got[[0, 2]]).all() and np.isfinite(got[1, :max(1, T - 2)]).all()
        if T > 1:
            assert np.isnan(got[1, T - 2:]).all()


@both
def test_infinite_scores_and_values_that_are_seen(q4):
    """NaN and infinities that a row sees reach it as in the formula."""
    ml = needs_gpu()
    c = Case(q4, [40, 70], 2, 4, 2, 128, 16, seed=12)
    if q4:
        c.cache[1][c.bt[0, 1], 0, 3, 2] = 0x7F     # a NaN key of head 0
        c.cache[3][c.bt[1, 2], 1, 5, 1] = 0x7F     # NaN values of head 1
    else:
        c.k[c.bt[0, 1], 3, 0, 40] = float("nan")
        c.v[c.bt[1, 2], 5, 1, 20] = float("inf")
    out, o = c.check(ml)
    got = out.float().cpu().numpy().reshape(2, 2, 4, 128)
    assert np.isnan(got[0, :, :2]).all() and np.isfinite(got[0, :, 2:]).all()
    assert (np.isnan(got[1, :, 2:, 16:32]).all() if q4 else np.isposinf(got[1, :, 2:, 20]).all())


@both
def test_strided_rows_other_columns_and_unaligned_views(q4):
    """q anywhere in wider rows of y; rows that no 16-byte load can reach."""
    ml = needs_gpu()
    for pad, q_col in ((64, 32), (37, 0), (40, 3), (7, 5)):
        Case(q4, [5, 100, 64], 3, 8, 2, 128, 16, seed=pad, pad=pad).check(ml, q_col=q_col)
    c = Case(q4, [5, 100, 64], 3, 8, 2, 128, 16, seed=4).device()
    buf = torch.empty(c.y_d.numel() + 1, dtype=torch.bfloat16, device="cuda")
    view = buf[1:].view_as(c.y_d)
    view.copy_(c.y_d)
    o, _, bound = c.oracle()
    got = c.call(ml, y=view).double().cpu().numpy().reshape(o.shape)
    assert np.all(np.abs(got - o) <= _tolerance(o, bound, 128, q4))


@both
def test_later_draft_steps(q4):
    """Draft step t0 sits t0 positions past the committed length."""
    ml = needs_gpu()
    for t0 in (1, 3, 100):
        Case(q4, [0, 31, 64, 100], 1, 8, 2, 128, 16, seed=t0, t0=t0).check(ml)


def test_units_of_the_4_bit_cache():
    ml = needs_gpu()
    Case(True, [40, 300], 3, 8, 2, 128, 16, unit=(0.37, 5.5)).check(ml)
    Case(True, [40, 300], 3, 8, 2, 64, 16, unit=(2.0 ** -6, 2.0 ** 9)).check(ml)


@both
@pytest.mark.parametrize("mag", [2.0 ** -30, 2.0 ** 40])
def test_queries_outside_fp16(q4, mag):
    """bf16 queries far below and above what fp16 holds."""
    ml = needs_gpu()
    c = Case(q4, [40, 300], 3, 8, 2, 128, 16, seed=1)
    c.y = (c.y.float() * mag).to(torch.bfloat16)
    c.check(ml, scale=0.088 / mag)


@both
def test_same_bits_every_time_and_from_a_graph(q4):
    """Repeated calls, calls on another stream, and a captured call give the same bits."""
    ml = needs_gpu()
    c = Case(q4, [3000, 17, 900, 64], 5, 10, 2, 128, 16, seed=8).device()
    ws = ml.Workspace(ml.attention_workspace_bytes(20, 5, 10, 2, 128))
    first = c.call(ml, ws=ws).clone()
    for _ in range(5):
        assert torch.equal(c.call(ml, ws=ws), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    c.call(ml, ws=ws, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, first)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(ml, ws=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert ws.status() == 0


@both
def test_cache_past_32_bit_offsets(q4):
    """Pages whose byte (and element) offsets pass 2^32."""
    ml = needs_gpu()
    H, D, bs = 8, 128, 16
    nb = 700000 if q4 else (1 << 18) + 4096          # 5.7e9 bytes of codes; 4.4e9 bf16 elements
    small = Case(q4, [200, 70], 3, 16, H, D, bs, seed=2)
    n = small.k.shape[0]
    move = nb - n                                    # the small cache's pages lie at the end of a large one
    big = []
    small.device()
    for c in small.c_d:
        t = torch.empty((nb,) + tuple(c.shape[1:]), dtype=c.dtype, device="cuda")
        t[move:] = c
        big.append(t)
    want = small.call(ml)
    small.c_d, small.bt_d = big, small.bt_d + move
    assert torch.equal(small.call(ml), want)
    if not q4:
        assert nb * bs * H * D > 1 << 32


@pytest.mark.parametrize("q4", [False, True], ids=["bf16", "q4"])
def test_no_rows(q4):
    ml = needs_gpu()
    c = Case(q4, [5], 1, 4, 2, 128, 16).device()
    assert c.call(ml, y=c.y_d[:0]).shape == (0, 512)


@both
def test_windowed_prompts_have_the_same_bits_every_time(q4):
    """Few sink tokens set a row's maximum before its window raises it: the
    outputs are rescaled while products are on their way."""
    ml = needs_gpu()
    c = Case(q4, [127, 1, 300], 129, 5, 1, 128, 32, seed=129)
    out, _ = c.check(ml, window=100, sinks=5)
    ws = ml.Workspace(ml.attention_workspace_bytes(3 * 129, 129, 5, 1, 128))
    for _ in range(50):
        assert torch.equal(c.call(ml, window=100, sinks=5, ws=ws), out)
    assert ws.status() == 0
