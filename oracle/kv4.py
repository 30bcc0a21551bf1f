"""The 4-bit pool on the CPU: quantiser, tile format, attention over it, and
page growth, each written out from its definition in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code
with the library.
"""
from __future__ import annotations

import numpy as np

TILE = 2912
KG, VG = 3, 2


def _next16(h, up):
    with np.errstate(over="ignore"):  # np.where evaluates it for values it does not take
        return np.nextafter(h, np.float16(np.inf if up else -np.inf), dtype=np.float16)


def fp16_down(x):
    """Largest fp16 value <= x (fp32), saturating at +-65504."""
    x = np.clip(x, np.float32(-65504), np.float32(65504))
    h = x.astype(np.float16)
    return np.where(h.astype(np.float32) > x, _next16(h, False), h)


def fp16_up(x):
    x = np.clip(x, np.float32(-65504), np.float32(65504))
    h = x.astype(np.float16)
    return np.where(h.astype(np.float32) < x, _next16(h, True), h)


def quantise(x):
    """x [..., 64 n] fp32 -> codes uint8 [..., 64 n], s, m fp16 [..., n]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 64)
    odd = ~np.isfinite(g).all(-1)
    g = np.where(odd[..., None], np.float32(0), g)
    m = fp16_down(g.min(-1))
    mf = m.astype(np.float32)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        s = fp16_up((g.max(-1) - mf) / np.float32(15))
        sf = s.astype(np.float32)[..., None]
        q = np.where(sf > 0, (g - mf[..., None]) / np.where(sf > 0, sf, np.float32(1)), np.float32(0))
    u = np.clip(np.rint(q), 0, 15).astype(np.uint8)
    nan = np.uint16(0x7FFF).view(np.float16)
    s, m = np.where(odd, nan, s).astype(np.float16), np.where(odd, nan, m).astype(np.float16)
    return u.reshape(x.shape), s, m


def dequantise(u, s, m):
    """fp64 values of codes [..., 64 n]."""
    g = u.reshape(*u.shape[:-1], -1, 64).astype(np.float64)
    return (m.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * g).reshape(u.shape)


def rope_fp32(k, cs):
    """k [T, H, 192] fp32, cs [T, 32, 2] fp32: rotate-half RoPE, each product and sum rounded to fp32."""
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = k[..., :32], k[..., 32:64]
    return np.concatenate([a * c - b * s, b * c + a * s, k[..., 64:]], -1).astype(np.float32)


def places(r):
    """Byte offsets of position r of a tile: K codes [192] (two dims share a byte), V codes [128], K scales [3],
    V scales [2], V minima [2], K minima [3]."""
    kc = [512 * (d // 64) + 64 * (r % 8) + 16 * (d % 64 // 16) + 8 * (r // 8) + d % 16 // 2 for d in range(192)]
    vc = [1536 + 512 * (d // 64) + 64 * (d % 64 // 8) + 16 * (r // 2 % 4) + 8 * (r // 8) + 4 * (d % 8 // 4)
          + 2 * (r % 2) + d % 4 // 2 for d in range(128)]
    c = 4 * (r // 2 % 4) + 2 * (r // 8) + r % 2
    return (np.array(kc), np.array(vc), np.array([2560 + 32 * g + 2 * c for g in range(3)]),
            np.array([2656 + 32 * g + 2 * c for g in range(2)]), np.array([2720 + 32 * g + 2 * c for g in range(2)]),
            np.array([2784 + 8 * r + 2 * g for g in range(3)]))


_PL = [places(r) for r in range(16)]


def _put16(tile, at, h):
    b = np.asarray(h, np.float16).view(np.uint16)
    tile[at] = b & 255
    tile[at + 1] = b >> 8


def _get16(tile, at):
    return (tile[..., at].astype(np.uint16) | (tile[..., at + 1].astype(np.uint16) << 8)).view(np.float16)


def write(data, blk, h, row, ku, ks, km, vu, vs, vm):
    """One position's codes and scales into data [blocks, H, tiles, 2912] uint8."""
    tile, r = data[blk, h, row // 16], row % 16
    kc, vc, aks, avs, avm, akm = _PL[r]
    tile[kc[0::2]] = ku[0::2] | (ku[1::2] << 4)
    tile[vc[0::2]] = vu[0::2] | (vu[1::2] << 4)
    for at, v in ((aks, ks), (avs, vs), (avm, vm), (akm, km)):
        _put16(tile, at, v)
    tile[2784 + 8 * r + 6:2784 + 8 * r + 8] = 0


def read(tiles):
    """Values of tiles [..., 2912]: K [..., 16, 192] and V [..., 16, 128] fp64."""
    K = np.zeros((*tiles.shape[:-1], 16, 192))
    V = np.zeros((*tiles.shape[:-1], 16, 128))
    hi = (np.arange(192) % 2 * 4).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        for r in range(16):
            kc, vc, aks, avs, avm, akm = _PL[r]
            K[..., r, :] = dequantise((tiles[..., kc] >> hi) & 15, _get16(tiles, aks), _get16(tiles, akm))
            V[..., r, :] = dequantise((tiles[..., vc] >> hi[:128]) & 15, _get16(tiles, avs), _get16(tiles, avm))
    return K, V


def sequence(data, table_row, h, n):
    """Values of positions 0..n-1 of one sequence and KV head, and which of them lie in a block of the pool."""
    bs = 16 * data.shape[2]
    nb = -(-n // bs)
    ids = np.asarray(table_row[:nb])
    ok = (ids >= 0) & (ids < data.shape[0])
    K, V = read(data[np.where(ok, ids, 0), h])
    return K.reshape(-1, 192)[:n], V.reshape(-1, 128)[:n], np.repeat(ok, bs)[:n]


def attend(q, pos, K, V, ok, cs, scale):
    """fp64 attention of q [G, 192] (raw) at position pos over keys 0..pos; cs [32, 2].  Returns out [G, 128] and, for
    error bounds, a = max_j scale * sum |q||k_j| [G] and w = sum_j p_j |v_j| [G, 128]."""
    q = np.asarray(q, np.float64)
    c, s = cs[:, 0].astype(np.float64), cs[:, 1].astype(np.float64)
    x = np.concatenate([q[:, :32] * c - q[:, 32:64] * s, q[:, 32:64] * c + q[:, :32] * s, q[:, 64:]], 1)
    n = pos + 1
    K, V, ok = K[:n], V[:n], ok[:n]
    K, V = K[ok], V[ok]
    if K.shape[0] == 0:
        return np.zeros((q.shape[0], 128)), np.zeros(q.shape[0]), np.zeros((q.shape[0], 128))
    S = x @ K.T * scale
    P = np.exp(S - S.max(1, keepdims=True))
    P /= P.sum(1, keepdims=True)
    return P @ V, (np.abs(x) @ np.abs(K).T).max(1) * abs(scale), P @ np.abs(V)


def grow(table, bs, num_blocks, seqs, lens, add, free, count, T):
    """kv_pages_grow in plain Python: (table, count, cu_rows, pos, row_seq, slots, flags) after the step."""
    table = table.copy()
    S, mb = table.shape
    n = len(seqs)
    flags = 0
    rows, need = [], 0
    for i in range(n):
        s, ln, ad = int(seqs[i]), int(lens[i]), int(add[i])
        if not 0 <= s < S:
            flags |= 2
            rows.append(0)
        elif ln < 0 or ad < 0 or ln + ad > mb * bs:
            flags |= 1
            rows.append(0)
        else:
            rows.append(ad)
            need += -(-(ln + ad) // bs) - -(-ln // bs)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    pos, rseq, slots = np.full(T, -1, np.int64), np.full(T, -1, np.int32), np.full(T, -1, np.int64)
    if cu[-1] > T or count < 0 or count > len(free) or need > count:
        flags |= 16 if cu[-1] > T else 64
        return table, count, np.zeros(n + 1, np.int32), pos, rseq, slots, flags
    k = 0
    for i in range(n):
        if rows[i] == 0:
            continue
        s, ln, ad = int(seqs[i]), int(lens[i]), int(add[i])
        for bi in range(-(-ln // bs), -(-(ln + ad) // bs)):
            b = int(free[count - 1 - k])
            k += 1
            if not 0 <= b < num_blocks:
                flags |= 4
                b = -1
            table[s, bi] = b
        for j in range(ad):
            p, r = ln + j, cu[i] + j
            b = int(table[s, p // bs])
            if not 0 <= b < num_blocks:
                flags |= 4
                b = -1
            pos[r], rseq[r] = p, s
            slots[r] = b * bs + p % bs if b >= 0 else -1
    return table, count - need, cu.astype(np.int32), pos, rseq, slots, flags
