"""The 8-bit pool on the CPU: scales, codes, tile format and attention over it,
each written out from its definition in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code
with the library.
"""
from __future__ import annotations

import numpy as np

TILE = 5136


def _bf16_floor(x):
    """Largest bf16 number <= x >= 0 (fp64), as fp64; the grid's step is 2^-7 of the power of two below, 2^-133 at least."""
    if x == 0:
        return 0.0, 2.0 ** -133
    e = max(int(np.floor(np.log2(x))), -126)
    if 2.0 ** e > x and e > -126:
        e -= 1
    step = 2.0 ** (e - 7)
    return float(np.floor(x / step) * step), step


def least_scale(a):
    """The least bf16 number s with 127 s >= a (a fp32, finite, >= 0), in exact arithmetic."""
    a = float(a)
    s, step = _bf16_floor(a / 127.0)
    while 127.0 * s < a:  # (products of 7 and 8 bits: exact)
        s += step
    while s > 0 and 127.0 * (s - step) >= a:
        s -= step
    return np.float32(s)


def codes(x, s):
    """rint(x / s) in fp32, ties to even; 0 where s is 0."""
    if s == 0:
        return np.zeros(np.shape(x), np.int64)
    return np.rint(np.asarray(x, np.float32) / np.float32(s)).astype(np.int64)


def rope_fp32(k, cs):
    """k [T, H, 192] fp32, cs [T, 32, 2] fp32: rotate-half RoPE, each product and sum rounded to fp32."""
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = k[..., :32], k[..., 32:64]
    with np.errstate(over="ignore", invalid="ignore"):
        return np.concatenate([a * c - b * s, b * c + a * s, k[..., 64:]], -1).astype(np.float32)


def places(r):
    """Byte offsets of position r of a tile: K codes [192], V codes [128]."""
    d, e = np.arange(192), np.arange(128)
    return 1024 * (d // 64) + 64 * r + d % 64, 16 * 192 + 512 * (e // 32) + 64 * (e % 32 // 4) + 16 * (r // 2 % 4) + 4 * (e % 4) + 2 * (r // 8) + r % 2


_PL = [places(r) for r in range(16)]


def scales(tile):
    return tile[5120:5128].copy().view(np.float32)


def masks(tile):
    return tile[5128:5132].copy().view(np.uint16)


def append(data, table_row, pos0, k, v):
    """One chunk's fp32 rows k [n, H, 192] (rotated), v [n, H, 128] (scaled) at positions pos0 .. of the sequence whose
    blocks are table_row, into data [blocks, H, tiles, 5136].  Tiles of no block of the pool are left out."""
    n, H = k.shape[:2]
    bs = 16 * data.shape[2]
    for m in range(pos0 // 16, (pos0 + n - 1) // 16 + 1):
        blk = int(table_row[16 * m // bs])
        if not 0 <= blk < data.shape[0]:
            continue
        first, last = max(16 * m, pos0), min(16 * m + 16, pos0 + n)
        ahead = first - 16 * m
        for h in range(H):
            tile = data[blk, h, (16 * m % bs) // 16]
            for which, x in ((0, k), (1, v)):
                rows = x[first - pos0:last - pos0, h]
                odd = ~np.isfinite(rows).all(-1)
                old = scales(tile)[which] if ahead else np.float32(0)
                need = least_scale(np.abs(rows[~odd]).max(initial=0))
                s = max(old, need)
                for r in range(ahead):  # (the same product in fp32 is exact: 7 and 8 bits)
                    at = _PL[r][which]
                    tile[at] = codes((tile[at].astype(np.int64) - 128).astype(np.float32) * old, s) + 128
                mask = int(masks(tile)[which]) & ((1 << ahead) - 1)
                for j in range(last - first):
                    tile[_PL[ahead + j][which]] = 128 if odd[j] else codes(rows[j], s) + 128
                    mask |= int(odd[j]) << (ahead + j)
                tile[5120 + 4 * which:5124 + 4 * which] = np.array([s], np.float32).view(np.uint8)
                tile[5128 + 2 * which:5130 + 2 * which] = np.array([mask], np.uint16).view(np.uint8)
            tile[5132:5136] = 0


def read(tiles):
    """Values of tiles [..., 5136]: K [..., 16, 192] and V [..., 16, 128] fp64."""
    out = []
    for which, width in ((0, 192), (1, 128)):
        x = np.zeros((*tiles.shape[:-1], 16, width))
        s = np.ascontiguousarray(tiles[..., 5120 + 4 * which:5124 + 4 * which]).view(np.float32)[..., 0].astype(np.float64)
        mask = np.ascontiguousarray(tiles[..., 5128 + 2 * which:5130 + 2 * which]).view(np.uint16)[..., 0]
        with np.errstate(invalid="ignore", over="ignore"):
            for r in range(16):
                x[..., r, :] = s[..., None] * (tiles[..., _PL[r][which]].astype(np.float64) - 128)
                x[..., r, :] = np.where((mask >> r & 1)[..., None] > 0, np.nan, x[..., r, :])
        out.append(x)
    return out


def sequence(data, table_row, h, n):
    """Values of positions 0..n-1 of one sequence and KV head, and which of them lie in a block of the pool."""
    bs = 16 * data.shape[2]
    nb = -(-n // bs)
    ids = np.asarray(table_row[:nb])
    ok = (ids >= 0) & (ids < data.shape[0])
    K, V = read(data[np.where(ok, ids, 0), h])
    return K.reshape(-1, 192)[:n], V.reshape(-1, 128)[:n], np.repeat(ok, bs)[:n]


def same(got, want, written):
    """Whether two pools agree on what means something: `written` has (block, tile) -> rows of a tile that are there;
    every other byte of them is free, and all bytes of other tiles agree."""
    for (blk, t), rows in written.items():
        for r in range(rows, 16):
            for at in _PL[r]:
                got[blk, :, t, at] = want[blk, :, t, at] = 0
    return np.array_equal(got, want)
