"""GPU parity of attention where 9 to 256 rows read a cache head together
(verify passes with grouped heads, chunks of prompts), with the float64 oracle.

The tolerances are those of test_gpu_attention: what is rounded is the same.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import needs_gpu
from tests.test_gpu_attention import BAD_SLOT, Case, _tolerance, both

pytestmark = pytest.mark.gpu

LENS = [0, 3, 60, 122, 127, 128, 129, 250, 256, 300, 640]


@both
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(9, 1), (3, 3), (17, 1), (6, 4), (8, 4), (11, 3), (9, 4), (8, 5), (12, 4), (7, 9), (16, 4),
                                 (13, 5), (33, 3), (128, 1), (25, 8), (64, 4)])
def test_rows_per_head(q4, D, T, G):
    """9 to 256 rows: below, at and past what a pass over the cache takes."""
    ml = needs_gpu()
    Case(q4, LENS, T, 2 * G, 2, D, 16, seed=T * G).check(ml)


@both
@pytest.mark.parametrize("bs", [1, 3, 8, 16, 20, 24, 33, 64, 128, 200, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(q4, D, bs):
    """Pages that do and do not divide a tile, and those that end inside one."""
    ml = needs_gpu()
    Case(q4, [5, 100, 131, 260, 390], 5, 15, 3, D, bs, seed=bs).check(ml)


@both
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (20, 0), (100, 4), (127, 0), (128, 16), (129, 130), (500, 300),
                                          (1000, 4)])
@pytest.mark.parametrize("T,G,D", [(5, 5, 128), (9, 4, 64), (40, 2, 128)])
def test_window_and_sinks(q4, window, sinks, T, G, D):
    ml = needs_gpu()
    Case(q4, [0, 1, 90, 127, 128, 200, 511, 900], T, 2 * G, 2, D, 16, seed=window).check(ml, window=window, sinks=sinks)


@both
@pytest.mark.parametrize("D", [64, 128])
def test_long_contexts_cut_over_the_gpu(q4, D):
    """Two requests over all SMs: every unit in many parts; and a long next to short ones."""
    ml = needs_gpu()
    Case(q4, [9000, 4097], 5, 10, 2, D, 16, seed=1).check(ml)
    Case(q4, [7000] + [10] * 40, 7, 8, 2, D, 16, seed=2).check(ml)


@both
def test_many_requests(q4):
    """More units than SMs, several to a CTA, some of which cuts go through."""
    ml = needs_gpu()
    g = np.random.default_rng(3)
    lens = g.integers(0, 700, 300).tolist()
    lens[7] = lens[100] = lens[299] = -1
    Case(q4, lens, 5, 12, 3, 128, 16, seed=3).check(ml)


@both
def test_more_requests_than_threads_count(q4):
    """The shares' prefix sums take several rounds."""
    ml = needs_gpu()
    lens = np.random.default_rng(4).integers(0, 40, 1500).tolist()
    Case(q4, lens, 7, 3, 1, 128, 16, seed=4).check(ml)


@both
@pytest.mark.parametrize("D", [64, 128])
def test_maxima_that_move(q4, D):
    """Scores of some hundreds of log2 units, growing along the context."""
    ml = needs_gpu()
    c = Case(q4, [50, 700, 1500], 6, 8, 2, D, 16, seed=5, spread=6.0)
    c.k = (c.k.float() * torch.linspace(0.1, 3.0, c.k.shape[0]).reshape(-1, 1, 1, 1)).to(torch.bfloat16)
    if q4:
        c.quantize()
    c.check(ml)


@both
@pytest.mark.parametrize("T,G,D", [(6, 4, 128), (9, 4, 64), (70, 1, 128), (130, 3, 128), (130, 3, 64)])
def test_values_that_are_not_finite_in_hidden_places(q4, T, G, D):
    """NaN and infinities after each row's own position, before its window and in
    the rest of the last page reach no row that does not see them."""
    ml = needs_gpu()
    c = Case(q4, [40, 200, 333], T, 2 * G, 2, D, 16, seed=6)
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
    assert np.isfinite(o[:T - 1]).any() and not np.isfinite(o).all()
    c.check(ml, window=30, sinks=1)


@both
def test_bad_pages(q4):
    """Pages that are not there are read as absent and reported."""
    ml = needs_gpu()
    c = Case(q4, [300, 500], 5, 10, 2, 128, 16, seed=7)
    c.bt[0, 3], c.bt[1, 20] = -1, 1 << 30
    c.check(ml, status=BAD_SLOT)


@both
def test_same_bits_every_time_and_from_a_graph(q4):
    ml = needs_gpu()
    c = Case(q4, [2000, 10, 900, 3000], 5, 20, 4, 128, 16, seed=8).device()
    ws = ml.Workspace(ml.attention_workspace_bytes(20, 5, 20, 4, 128))
    first = c.call(ml, ws=ws).clone()
    out = torch.empty_like(first)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        c.call(ml, ws=ws, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            c.call(ml, ws=ws, out=out)
    torch.cuda.current_stream().wait_stream(stream)
    for _ in range(20):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)


@both
def test_negative_scale_and_large_and_small_queries(q4):
    ml = needs_gpu()
    c = Case(q4, [100, 260], 5, 10, 2, 128, 16, seed=9)
    c.check(ml, scale=-0.1)
    c.y = (c.y.float() * 2.0 ** -40).to(torch.bfloat16)
    c.check(ml, scale=2.0 ** 36)


@both
@pytest.mark.parametrize("T,G,D,M", [(5, 5, 128, 11), (5, 5, 64, 14), (8, 8, 64, 17), (40, 4, 128, 82), (40, 4, 64, 121),
                                     (300, 2, 128, 700), (300, 2, 64, 601), (3, 2, 128, 4), (5, 5, 128, 5)])
def test_a_last_request_in_part_and_requests_without_rows(q4, T, G, D, M):
    """M rows that end within a request: its first rows alone; later requests have none."""
    ml = needs_gpu()
    c = Case(q4, [130, 300, 77, 500], T, 2 * G, 2, D, 16, seed=M)
    ws = ml.Workspace(ml.attention_workspace_bytes(M, T, 2 * G, 2, D))
    got = c.device().call(ml, y=c.y_d[:M].contiguous(), ws=ws).double().cpu().numpy().reshape(M, 2 * G, D)
    c.y = c.y[:M]
    o, st, bound = c.oracle()
    assert st == 0 and ws.status() == 0
    assert (np.abs(got - o) <= _tolerance(o, bound, D, q4)).all()
