"""The microscaled 4-bit form and the expert routing in plain NumPy fp64 (test infrastructure only).

e2m1 numbers are rounded by their step (0.5 below 2, 1 below 4, 2 above), half to even, which is the
even code; e4m3 by its step of an eighth of the binade. Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

BLOCK = {"mx": 32, "nv": 16}


def e2m1_round(y):
    """Nearest e2m1 number (ties to the even code), saturating at 6."""
    m = np.abs(y)
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    return np.copysign(np.minimum(np.rint(m / step) * step, 6.0), y)


def e2m1_code(v):
    """Code of an e2m1 number: the place in 0, 0.5, 1, 1.5, 2, 3, 4, 6, plus 8 where negative (a
    negative zero has code 8)."""
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.searchsorted(grid, np.abs(v)) + 8 * np.signbit(v)


def e4m3_round(a):
    """Nearest e4m3 number (ties to even) of a >= 0, saturating at 448."""
    a = np.minimum(a, 448.0)
    _, e = np.frexp(np.maximum(a, 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.rint(a / step) * step


def e4m3_byte(s):
    """Byte of a nonnegative e4m3 number."""
    m, e = np.frexp(np.maximum(s, 2.0 ** -9))
    normal = ((e - 1 + 7) << 3) + np.rint((2 * m - 1) * 8).astype(int)
    return np.where(s < 2.0 ** -6, np.rint(s * 512).astype(int), normal).astype(np.uint8)


def quantise(x, fmt, g=None):
    """(values fp64 (rows, cols), codes (rows, cols), scale bytes (rows, blocks)) of fp32 x."""
    rows, cols = x.shape
    B = BLOCK[fmt]
    xb = np.zeros((rows, -(-cols // B) * B))
    xb[:, :cols] = x
    xb = xb.reshape(rows, -1, B)
    a = np.abs(xb).max(-1)
    if fmt == "mx":
        _, e = np.frexp(a)
        byte = np.where(a > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
        s = np.where(a > 0, np.ldexp(1.0, byte - 127), 0.0)
        d = s
    else:
        # the block's maximum over 6 g and its scale times g are each rounded to fp32 once
        s = e4m3_round((np.float32(a) / (np.float32(6) * np.float32(g))).astype(np.float64))
        byte = e4m3_byte(s)
        d = np.float64(np.float32(s) * np.float32(g))
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = np.where(d[..., None] > 0, (xb / np.where(d > 0, d, 1)[..., None]).astype(np.float32), 0.0)
    v = e2m1_round(y)
    return ((v * d[..., None]).reshape(rows, -1)[:, :cols], e2m1_code(v).reshape(rows, -1)[:, :cols].astype(np.uint8),
            byte.astype(np.uint8))


def pack_codes(codes):
    rows, cols = codes.shape
    c = np.zeros((rows, -(-cols // 32) * 32), np.uint8)
    c[:, :cols] = codes
    return c[:, 0::2] | (c[:, 1::2] << 4)


def tile_scales(byte, cols, fmt):
    """(rows, blocks) -> (row tiles, block tiles, 512), zeros outside the matrix."""
    rows, blocks = byte.shape
    tk = -(-cols // (4 * BLOCK[fmt]))
    out = np.zeros((-(-rows // 128), tk, 512), np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    out[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte
    return out


def untile_scales(tiles, rows, blocks):
    r, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    return tiles[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def values(codes, byte, fmt, g=1.0):
    """fp64 values of codes (rows, cols) and scale bytes (rows, blocks)."""
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    v = grid[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    if fmt == "mx":
        s = np.ldexp(1.0, byte.astype(int) - 127)
    else:
        e, f = byte.astype(int) >> 3, byte.astype(int) & 7
        s = np.where(e > 0, np.ldexp(1 + f / 8, e - 7), f / 512) * g
    return v * np.repeat(s, BLOCK[fmt], axis=1)[:, :codes.shape[1]]


def route(ids, experts):
    """(offsets, src, pos) of ids (tokens, top), slot by slot."""
    flat = ids.reshape(-1)
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(i)
    offsets = np.concatenate(([0], np.cumsum([len(v) for v in lists])))
    order = [i for v in lists for i in v]
    src = np.full(flat.size, -1)
    src[:len(order)] = order
    pos = np.full(flat.size, -1)
    pos[order] = np.arange(len(order))
    return offsets, src, pos.reshape(ids.shape)
