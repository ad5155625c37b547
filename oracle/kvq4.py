"""Oracle for the KV cache in 4 bits: quantising a pass's K and V rows as they
are written and reading positions back (numpy; exact rounding to E2M1 and E4M3
from their definitions).

Test infrastructure only (see the package docstring).

The pages describe one paged cache for both passes and no narrower format.  The
readings taken: groups of 16 values along a head's D; E2M1 codes (bias 1: 0,
.5, 1, 1.5, 2, 3, 4, 6 and a sign bit, the even element in a byte's low half);
one E4M3 scale a group; a value is code * scale * unit with one fp32 unit per
cache.  scale = E4M3(amax / (6 unit)), code = E2M1(v / (scale unit)), the
quotients in fp32, both roundings to nearest even and saturating.  A group
whose scale is 0 has codes 0; a NaN in a group makes its scale NaN.  Rows,
positions, invalid slots and unused requests follow oracle.kvcache.
"""
from __future__ import annotations

import numpy as np

from oracle.fp8 import e4m3_decode, e4m3_round
from oracle.kvcache import BAD_SLOT, slot_of

GROUP = 16
E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_round(v) -> np.ndarray:
    """E2M1 codes (0..15, bit 3 the sign) of fp32 values: nearest, ties to the
    even code, saturating at 6.  NaN is not defined here (its group reads as NaN
    whatever the codes): code 0."""
    x = np.asarray(v, dtype=np.float32).astype(np.float64)
    a = np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300))
    d = np.abs(a[..., None] - E2M1_VALUES)
    d[a > 6.0] = np.arange(8, 0, -1)                  # saturation
    best = d.min(-1, keepdims=True)
    near = d == best                                  # two on a tie: take the even one
    first = near.argmax(-1)
    tie = near.sum(-1) == 2
    code = np.where(tie & (first % 2 == 1), first + 1, first)
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 8, 0)).astype(np.uint8)


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * E2M1_VALUES[c & 7]


def quantize(v, unit: float = 1.0):
    """Values [..., D] (bf16-valued) -> (packed codes uint8 [..., D/2], E4M3
    scale codes uint8 [..., D/16])."""
    g = np.asarray(v, dtype=np.float32)
    g = g.reshape(g.shape[:-1] + (-1, GROUP))
    unit = np.float32(unit)
    nan = np.isnan(g).any(-1)
    with np.errstate(all="ignore"):
        amax = np.where(nan, np.float32(np.nan), np.abs(g).max(-1)).astype(np.float32)
        sc = e4m3_round(amax / (np.float32(6.0) * unit))
        s = (e4m3_decode(sc).astype(np.float32) * unit)[..., None]
        code = np.where(s == 0, 0, e2m1_round((g / s).astype(np.float32)))
    code = code.reshape(code.shape[:-2] + (-1,)).astype(np.uint8)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), sc


def dequantize(codes, scales, unit: float = 1.0) -> np.ndarray:
    """Float64 values of packed codes and E4M3 scales."""
    c = np.asarray(codes, dtype=np.uint8)
    full = np.stack((c & 15, c >> 4), -1).reshape(c.shape[:-1] + (-1,))
    v = e2m1_decode(full)
    return v * np.repeat(e4m3_decode(scales), GROUP, -1) * np.float64(np.float32(unit))


def kv_write_q4(y, k_col, v_col, H, D, block_table, seq_len, rows_per_req, t0, cache, k_unit=1.0, v_unit=1.0):
    """y fp32 (bf16-valued) [M, ld]; cache = (k_codes, k_scales, v_codes,
    v_scales).  Returns (new cache, status)."""
    cache = [np.array(c, copy=True) for c in cache]
    nb, bs = cache[0].shape[0], cache[0].shape[2]
    status = 0
    for m in range(y.shape[0]):
        b, t = divmod(m, rows_per_req)
        if int(seq_len[b]) < 0:
            continue
        where = slot_of(block_table, seq_len, b, t0 + t, bs, nb)
        if where is None:
            status |= BAD_SLOT
            continue
        blk, off = where
        for i, (col, unit) in enumerate(((k_col, k_unit), (v_col, v_unit))):
            c, s = quantize(y[m, col:col + H * D].reshape(H, D), unit)
            cache[2 * i][blk, :, off], cache[2 * i + 1][blk, :, off] = c, s
    return cache, status


def kv_read_q4(cache, block_table, start, end, rows, k_unit=1.0, v_unit=1.0):
    """(K, V) float64 [B, rows, H, D] and the status."""
    nb, H, bs, half = cache[0].shape
    B = len(start)
    out = [np.zeros((B, rows, H, 2 * half)) for _ in range(2)]
    status = 0
    for b in range(B):
        for t in range(rows):
            if int(start[b]) < 0 or int(start[b]) + t >= int(end[b]):
                continue
            where = slot_of(block_table, start, b, t, bs, nb)
            if where is None:
                status |= BAD_SLOT
                continue
            blk, off = where
            for i, unit in enumerate((k_unit, v_unit)):
                out[i][b, t] = dequantize(cache[2 * i][blk, :, off], cache[2 * i + 1][blk, :, off], unit)
    return out[0], out[1], status
