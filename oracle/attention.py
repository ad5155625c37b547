"""Oracle for attention over the paged cache: float64 softmax over the
positions each row sees (numpy).

Test infrastructure only (see the package docstring).

Both passes of the InvisibleLoRA abstract read one cache; the abstract gives no
formula for the attention itself, so the usual one is taken: o = sum_j p_j v_j
with p the softmax of scale * q . k_j over the positions seen.  Row m is request
b = m // rows_per_req at position p = seq_len[b] + t0 + m % rows_per_req; it
sees j <= p, with window > 0 of those only j > p - window or j < sinks, and
never a position whose slot lies outside the cache or the request's table
(status bit 7).  A row that sees nothing is zeros, as is every row of an unused
request slot.  Hidden positions are left out of the sums, so what they hold has
no effect.
"""
from __future__ import annotations

import numpy as np

from oracle.kvcache import BAD_SLOT


def visible(pos: int, window: int, sinks: int) -> np.ndarray:
    """The positions a row at `pos` sees, in order."""
    j = np.arange(pos + 1)
    if window <= 0:
        return j
    return j[(j > pos - window) | (j < sinks)]


def attention(q, keys_of, B, rows_per_req, Hq, H, D, block_table, block_size, num_blocks, seq_len, t0, scale,
              window=0, sinks=0):
    """q [M, Hq, D] float64; keys_of(blk, off, h) -> (k, v) float64 arrays for
    arrays of blocks and offsets ([n, D] each).

    Returns (o [M, Hq, D], status, bound) with bound a dict of float64 arrays
    per output row [M, Hq] that error bounds need: "A" [M, Hq, D] the weighted
    sum of |v|, "S" the largest scale * sum |q k|, "n" the positions seen,
    "qk" scale * max|q| * max|k|, "v" [M, Hq, D] the largest |v|."""
    M = q.shape[0]
    o = np.zeros((M, Hq, D))
    A, vmax = np.zeros((M, Hq, D)), np.zeros((M, Hq, D))
    S, n, qk = np.zeros((M, Hq)), np.zeros((M, Hq)), np.zeros((M, Hq))
    status, G = 0, Hq // H
    for m in range(M):
        b, t = divmod(m, rows_per_req)
        if int(seq_len[b]) < 0:
            continue
        j = visible(int(seq_len[b]) + t0 + t, window, sinks)
        inside = j < block_table.shape[1] * block_size
        page = np.where(inside, block_table[b, np.minimum(j // block_size, block_table.shape[1] - 1)], -1)
        ok = inside & (page >= 0) & (page < num_blocks)
        if not ok.all():
            status |= BAD_SLOT
        j, page = j[ok], page[ok]
        if len(j) == 0:
            continue
        for h in range(H):
            k, v = keys_of(page, j % block_size, h)
            for hq in range(h * G, (h + 1) * G):
                with np.errstate(all="ignore"):
                    z = scale * (k @ q[m, hq])
                    p = np.exp(z - z.max())
                    o[m, hq] = (p @ v) / p.sum()
                    A[m, hq] = (p @ np.abs(v)) / p.sum()
                    S[m, hq] = abs(scale) * (np.abs(k) @ np.abs(q[m, hq])).max()
                    qk[m, hq] = abs(scale) * np.abs(q[m, hq]).max() * np.abs(k).max()
                    vmax[m, hq] = np.abs(v).max(0)
                n[m, hq] = len(j)
    return o, status, {"A": A, "S": S, "n": n, "qk": qk, "v": vmax}
