"""GPU parity of attention over many rows and enough (request, cache head) units
to fill the GPU, with the float64 oracle.

The tolerances are those of test_gpu_attention: what is rounded is the same.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import needs_gpu
from tests.test_gpu_attention import BAD_SLOT, Case, both

pytestmark = pytest.mark.gpu


@both
@pytest.mark.parametrize("T,G,D,B", [(130, 2, 128, 5), (65, 4, 128, 5), (300, 1, 128, 12), (33, 4, 64, 11), (65, 2, 64, 12),
                                     (130, 2, 64, 6), (261, 1, 64, 12)])
def test_rows(q4, T, G, D, B):
    """Row tiles full and in part, one and several a unit."""
    ml = needs_gpu()
    lens = [0, 1, 127, 128, 129, 60, 255, 256, 300, 5, 64, 190][:B]
    Case(q4, lens, T, 8 * G, 8, D, 16, seed=T).check(ml)


@both
@pytest.mark.parametrize("bs", [1, 3, 8, 20, 33, 64, 128, 200])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(q4, D, bs):
    """Pages brought in boxes and in pieces."""
    ml = needs_gpu()
    Case(q4, [5, 100, 131, 260, 17, 0], 66, 32, 8, D, bs, seed=bs).check(ml)


@both
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (128, 16), (129, 130), (1000, 4)])
@pytest.mark.parametrize("T,D", [(70, 128), (33, 64)])
def test_window_and_sinks(q4, window, sinks, T, D):
    ml = needs_gpu()
    Case(q4, [0, 90, 127, 128, 511, 300, 1, 77, 130, 50], T, 32, 8, D, 16, seed=window).check(ml, window=window, sinks=sinks)


@both
@pytest.mark.parametrize("T,D", [(70, 128), (33, 64), (130, 64)])
def test_values_that_are_not_finite_in_hidden_places(q4, T, D):
    ml = needs_gpu()
    c = Case(q4, [40, 200, 133, 0, 64, 127, 90, 3, 15, 31], T, 32, 8, D, 16, seed=6)
    page = lambda b, p: int(c.bt[b, p // 16])  # noqa: E731
    for b, L in enumerate(c.seq):
        last = int(L) + T - 1
        for p in range(last, (last // 16 + 1) * 16):        # only the last row sees `last`
            if q4:
                c.cache[3][page(b, p), :, p % 16] = 0x7F
            else:
                c.v[page(b, p), p % 16] = float("nan") if p % 2 else float("inf")
        if q4:
            c.cache[3][page(b, 2), :, 2] = 0x7F
        else:
            c.v[page(b, 2), 2, :, ::3] = float("-inf")
    c.check(ml)
    _, o = c.check(ml, window=20)
    assert np.isfinite(o).any() and not np.isfinite(o).all()


@both
@pytest.mark.parametrize("D", [64, 128])
def test_maxima_that_move_and_bad_pages(q4, D):
    ml = needs_gpu()
    c = Case(q4, [50, 700, 300, 10, 90, 128], 66, 32, 8, D, 16, seed=5, spread=6.0)
    c.k = (c.k.float() * torch.linspace(0.1, 3.0, c.k.shape[0]).reshape(-1, 1, 1, 1)).to(torch.bfloat16)
    if q4:
        c.quantize()
    c.check(ml)
    c.bt[0, 3], c.bt[1, 20] = -1, 1 << 30
    c.check(ml, status=BAD_SLOT)


@both
@pytest.mark.parametrize("D", [64, 128])
def test_same_bits_every_time(q4, D):
    ml = needs_gpu()
    c = Case(q4, [2000, 10, 900, 300, 0, 128], 66, 32, 8, D, 16, seed=8).device()
    ws = ml.Workspace(ml.attention_workspace_bytes(6 * 66, 66, 32, 8, D))
    first = c.call(ml, ws=ws).clone()
    for _ in range(20):
        assert torch.equal(c.call(ml, ws=ws), first)


@both
def test_unused_and_partial_requests(q4):
    ml = needs_gpu()
    c = Case(q4, [100, -1, 260, 33, -1, 64], 66, 32, 8, 128, 16, seed=9)
    c.check(ml)
