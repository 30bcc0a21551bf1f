"""The 4-bit pool on the GPU: the append's bytes against the oracle's bit for
bit, the decode against fp64 attention over the values the codes stand for,
the unpack bit for bit, page growth against plain Python, and a run of them
together with the bf16 calls they stand beside."""
import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import kv4 as o4

from kvr_cases import SCALE

pytestmark = pytest.mark.gpu
DEV = "cuda"
VS = 0.707


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sinks_kv_ring_gb300 import build
    build.build()
    kvr.device_status(reset=True)
    yield


@pytest.fixture(scope="module")
def table():
    return kvr.rope_table(1e7, 1 << 17)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _kv(gen, T, hkv, shift=0.0):
    k = torch.randn(T, hkv, 192, generator=gen, device=DEV)
    k[..., 64:] += shift * torch.randn(1, hkv, 128, generator=gen, device=DEV)
    return k.bfloat16(), torch.randn(T, hkv, 128, generator=gen, device=DEV).bfloat16()


def _pool(gen, S, hkv, max_ctx, bs, fill=0xFF, spare=3):
    """A pool with its blocks in random order and every byte `fill` (0xFF: NaN scales and minima wherever nothing is
    written)."""
    mb = -(-max_ctx // bs)
    nb = S * mb + spare
    ids = torch.randperm(nb, generator=gen, device=DEV)[:S * mb].to(torch.int32).reshape(S, mb)
    data = torch.full((nb, hkv, bs // 16, kvr.KV4_TILE), fill, dtype=torch.uint8, device=DEV)
    return kvr.Kv4Layout(data, ids.contiguous())


def _append(pool, k, v, seq, lo, table):
    T = k.shape[0]
    pos = torch.arange(lo, lo + T, device=DEV)
    kvr.kv4_append_rope(k, v, pos, torch.full((T,), seq, dtype=torch.int32, device=DEV), table, VS, pool)


def _ints(v, t):
    return torch.tensor(v, dtype=t, device=DEV)


def _want_bytes(pool, k, v, places, pos, table):
    """The pool's bytes after the append, by the oracle; places[t] = (block, row) or None."""
    data = pool.data.cpu().numpy().copy()
    cs = table[pos.clamp(0, table.shape[0] - 1)].cpu().numpy()
    kf = o4.rope_fp32(k.float().cpu().numpy(), cs)
    with np.errstate(over="ignore", invalid="ignore"):
        vf = v.float().cpu().numpy() * np.float32(VS)
        ku, ks, km = o4.quantise(kf)
        vu, vs, vm = o4.quantise(vf)
    for t, pl in enumerate(places):
        if pl is not None:
            for h in range(k.shape[1]):
                o4.write(data, pl[0], h, pl[1], ku[t, h], ks[t, h], km[t, h], vu[t, h], vs[t, h], vm[t, h])
    return data


# -- append --------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("by_slot", [False, True])
@pytest.mark.parametrize("T,hkv,bs", [(1, 1, 16), (3, 2, 64), (37, 3, 48), (64, 4, 16), (130, 8, 128), (257, 5, 1024)])
def test_append_bytes(table, T, hkv, bs, by_slot):
    gen = _gen(100 + T)
    S = 3
    pool = _pool(gen, S, hkv, 2048, bs, fill=0xEE)
    k, v = _kv(gen, T, hkv, 2.0)
    # distinct (sequence, position) pairs in random order
    pick = torch.randperm(S * 2048, generator=gen, device=DEV)[:T]
    seq, pos = (pick // 2048).to(torch.int32), pick % 2048
    blk = pool.block_table[seq.long(), pos // bs].long()
    want = _want_bytes(pool, k, v, list(zip(blk.tolist(), (pos % bs).tolist())), pos, table)
    if by_slot:
        kvr.kv4_append_rope(k, v, pos, None, table, VS, pool, slots=blk * bs + pos % bs)
    else:
        kvr.kv4_append_rope(k, v, pos, seq, table, VS, pool)
    assert np.array_equal(pool.data.cpu().numpy(), want)
    assert kvr.device_status() == 0


def test_append_corner_groups(table):
    gen = _gen(7)
    T, hkv = 12, 2
    pool = _pool(gen, 1, hkv, 64, 16, fill=0)
    k, v = _kv(gen, T, hkv)
    k[0, 0, 64:128] = 3.0                      # constant, and held by fp16
    k[1, 0, 64:128] = 0.1                      # constant, not held by fp16's grid of its own
    k[2, 1, 130] = float("nan")
    k[3, 1, 70] = float("inf")
    v[4, 0, 5] = float("-inf")
    v[5, 1, 64:] = 0.0
    v[6, 0] *= 1e-7                            # below fp16's normal range
    v[7, 0] *= 1e30                            # past fp16
    k[8, 0, 64:128] = torch.linspace(-3e38, 3e38, 64, device=DEV).bfloat16()
    k[9, 1, 64:128] = -0.0
    k[10, 0, :64] = 1e5                        # rotated, past fp16
    v[11, 1, :64] = torch.arange(64, device=DEV).bfloat16() * 0.5 / VS  # many values near half steps
    pos = torch.arange(T, device=DEV)
    want = _want_bytes(pool, k, v, [(int(pool.block_table[0, 0]), t) for t in range(T)], pos, table)
    _append(pool, k, v, 0, 0, table)
    got = pool.data.cpu().numpy()
    # a minimum of zeros of both signs may keep either sign: compare the bits, but for the sign of a zero fp16 minimum
    for r in range(16):
        *_, avm, akm = o4.places(r)
        for at in list(avm) + list(akm):
            for d in (got, want):
                hi, lo = d[..., at + 1], d[..., at]
                hi[(hi == 0x80) & (lo == 0)] = 0
    assert np.array_equal(got, want)


def test_append_value_products_are_rounded(table):
    """Values whose code hangs on the rounding of value times value scale: a product added without it falls on the other
    side of a half step."""
    rng = np.random.default_rng(1)
    vs = np.float32(VS)

    def bf16(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()

    n = 400000
    x = np.zeros((n, 64), np.float32)
    x[:, 0], x[:, 1] = bf16(-1 - 3 * rng.random(n)), bf16(1 + 3 * rng.random(n))
    with np.errstate(divide="ignore", invalid="ignore"):
        _, s, m = (a.astype(np.float32) if a.dtype != np.uint8 else a for a in o4.quantise(x * vs))
        v = bf16((m + s * (np.arange(15, dtype=np.float32) + np.float32(0.5))) / vs)
        rounded = (v * vs - m) / s
        fused = (v.astype(np.float64) * np.float64(vs) - m).astype(np.float32) / s
    hit = (np.rint(rounded) != np.rint(fused)) & (v > x[:, :1]) & (v < x[:, 1:2])
    rows = np.flatnonzero(hit.any(1))
    assert len(rows) >= 16
    rows = rows[:16]
    x[rows, 2:17] = np.where(hit[rows], v[rows], 0)
    vals = torch.from_numpy(x[rows]).bfloat16().to(DEV)                     # [16, 64]
    v1 = torch.cat([vals, vals.flip(1)], 1)[:, None].expand(16, 2, 128).contiguous()
    k1, _ = _kv(_gen(9), 16, 2)
    small = _pool(_gen(4), 1, 2, 16, 16, fill=0)
    pos = torch.arange(16, device=DEV)
    want = _want_bytes(small, k1, v1, [(int(small.block_table[0, 0]), t) for t in range(16)], pos, table)
    _append(small, k1, v1, 0, 0, table)
    assert np.array_equal(small.data.cpu().numpy(), want)
    many = 2200                                                             # 70,400 pairs: the same values 2200 times
    big = _pool(_gen(4), many, 2, 16, 16, fill=0)
    kvr.kv4_append_rope(k1.repeat(many, 1, 1), v1.repeat(many, 1, 1), pos.repeat(many),
                        torch.arange(many, device=DEV).repeat_interleave(16).to(torch.int32), table, VS, big)
    tile = small.data[small.block_table[0, 0].long()]
    assert torch.equal(big.data[big.block_table[:, 0].long()], tile.expand(many, *tile.shape))


@pytest.mark.parametrize("hkv,by_slot,scale", [(1, False, VS), (2, True, VS), (3, False, -VS), (5, True, -1.0), (8, False, VS)])
def test_append_many_as_few(table, hkv, by_slot, scale):
    """A call of many (token, KV head) pairs writes the bytes that calls of a few tokens write, and says the same of the
    tokens it cannot write."""
    gen = _gen(300 + hkv)
    T, bs, S = 66001 // hkv + 1, 48, 4
    mb = -(-T // (S * bs)) + 1
    pools = [_pool(_gen(5), S, hkv, mb * bs, bs, fill=0x3C) for _ in range(2)]
    k, v = _kv(gen, T, hkv, 2.0)
    hit = torch.randint(0, T, (60,), generator=gen, device=DEV)
    k[hit[:10], :, 3] = float("nan")
    k[hit[10:20], -1, 70] = float("inf")
    k[hit[20:30], 0, 64:128] *= 1e30
    k[hit[30:35]] = 1.5
    v[hit[35:45], -1] *= 1e6
    v[hit[45:50], 0, 127] = float("-inf")
    v[hit[50:60]] = 0.0
    pick = torch.randperm(S * mb * bs, generator=gen, device=DEV)[:T]
    seq, pos = (pick // (mb * bs)).to(torch.int32), pick % (mb * bs)
    slots = pools[0].block_table[seq.long(), pos // bs].long() * bs + pos % bs
    off = torch.randint(0, T, (40,), generator=gen, device=DEV)
    seq[off[:10]], slots[off[:10]] = -1, -1
    seq[off[10:20]], slots[off[10:20]] = S, 1 << 40
    pos[off[20:30]] = 1 << 17
    pos[off[30:]] = -7
    step = 997

    def run(pool, lo, hi):
        kvr.kv4_append_rope(k[lo:hi], v[lo:hi], pos[lo:hi], None if by_slot else seq[lo:hi], table, scale, pool,
                            slots=slots[lo:hi] if by_slot else None)

    run(pools[0], 0, T)
    status = kvr.device_status()
    for lo in range(0, T, step):
        run(pools[1], lo, min(lo + step, T))
    assert kvr.device_status() == status == kvr.DEV_BAD_POS | (kvr.DEV_BAD_BLOCK if by_slot else kvr.DEV_BAD_SEQ)
    assert torch.equal(pools[0].block_table, pools[1].block_table)
    assert torch.equal(pools[0].data, pools[1].data)


def test_append_padding_and_flags(table):
    gen = _gen(8)
    T, hkv, bs = 8, 2, 32
    pool = _pool(gen, 2, hkv, 128, bs, fill=0x55)
    pool.block_table[1, 2] = -1
    pool.block_table[1, 3] = pool.num_blocks
    k, v = _kv(gen, T, hkv)
    before = pool.data.clone()

    def run(pos, seq=None, slots=None):
        kvr.kv4_append_rope(k, v, _ints(pos, torch.int64), None if seq is None else _ints(seq, torch.int32), table, VS,
                            pool, slots=None if slots is None else _ints(slots, torch.int64))
        return kvr.device_status()

    big = 1 << 40
    assert run([-1] * T, [-1] * T) == 0                       # padding: skipped without a flag
    assert run([-1] * T, slots=[-1, -2, -big, -1, -1, -1, -1, -1]) == 0
    assert torch.equal(pool.data, before)
    assert run([-1, 1 << 17, -5, big, -1, -1, -1, -1], [0, 0, 1, 1, -1, -1, -1, -1]) == kvr.DEV_BAD_POS
    assert run([5] * T, [2, -2, 9, 2 ** 31 - 1, -1, -1, -1, -1]) == kvr.DEV_BAD_SEQ
    assert run([64, 96, 128, 1000, 0, 0, 0, 0], [1, 1, 1, 0, -1, -1, -1, -1]) == kvr.DEV_BAD_BLOCK
    nslot = pool.num_blocks * bs
    assert run([0] * T, slots=[nslot, big, nslot + 5] + [-1] * 5) == kvr.DEV_BAD_BLOCK
    assert run([-3, 1 << 17] + [0] * 6, slots=[0, 1] + [-1] * 6) == kvr.DEV_BAD_POS
    assert torch.equal(pool.data, before)
    # a good token beside bad ones is written
    assert run([40, -1, 7, 0, 0, 0, 0, 0], [0, 0, 5, -1, -1, -1, -1, -1]) == kvr.DEV_BAD_POS | kvr.DEV_BAD_SEQ
    want = _want_bytes(kvr.Kv4Layout(before, pool.block_table), k, v,
                       [(int(pool.block_table[0, 1]), 8)] + [None] * 7, _ints([40] * T, torch.int64), table)
    assert np.array_equal(pool.data.cpu().numpy(), want)


# -- decode --------------------------------------------------------------------------------------------------------------

def _check_decode(got, q, pos, seq, pool, table, what=""):
    """Every row against fp64.  The output is rounded by half a bf16 step, 2^-8 |o| at most.  A score moves by at most
    2^-11 sum |q||k| for the rounding of the rotated q to fp16, and by less than as much again for everything held in
    fp32 or in two fp16 parts: 2^-10 sum |q||k|, which moves a weight by twice that at most (its own score's and the
    sum's part).  A weight is rounded to fp16 twice, 2^-11 each, and their sum with the minima once: 2^-10 of sum p |v|,
    where |v| counts the code part and the minimum apart, at most 3 |v|_max of the group.  And the bar of the bf16
    decode, per row."""
    data, bt = pool.data.cpu().numpy(), pool.block_table.cpu().numpy()
    cs = table.cpu().numpy()
    G = q.shape[1] // pool.num_kv_heads
    qf, g = q.float().cpu().numpy(), got.double().cpu().numpy()
    cache = {}
    for b, (p, s) in enumerate(zip(pos, seq)):
        for h in range(pool.num_kv_heads):
            if (s, h) not in cache:
                n = max(pp for pp, ss in zip(pos, seq) if ss == s) + 1
                cache[s, h] = o4.sequence(data, bt[s], h, n)
            K, V, ok = cache[s, h]
            hs = slice(h * G, (h + 1) * G)
            want, a, w = o4.attend(qf[b, hs], p, K, V, ok, cs[p], SCALE)
            err = np.abs(g[b, hs] - want)
            vmax = np.abs(V[:p + 1][ok[:p + 1]]).max() if ok[:p + 1].any() else 0.0
            tol = 2.0 ** -8 * np.abs(want) + 2 * 2.0 ** -10 * a[:, None] * w + 2.0 ** -10 * (w + 3 * vmax)
            assert np.all(err <= tol), f"{what} row {b} head {h}: {np.max(err - tol):.3e} over"
            rel = np.sqrt((err ** 2).mean(1) / np.maximum((want ** 2).mean(1), 1e-30))
            assert rel.max() <= 1e-2, f"{what} row {b} head {h}: rel RMS {rel.max():.3e}"


def _filled(gen, lens, hkv, bs, table, shift=0.0, max_ctx=None):
    pool = _pool(gen, len(lens), hkv, max_ctx or max(lens), bs)
    for s, n in enumerate(lens):
        k, v = _kv(gen, n, hkv, shift)
        _append(pool, k, v, s, 0, table)
    return pool


@pytest.mark.parametrize("bs", [16, 48, 64, 256])
@pytest.mark.parametrize("G", [1, 3, 8, 13, 16])
def test_decode_ragged(table, G, bs):
    gen = _gen(1000 + 10 * G + bs)
    hkv = 2
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 513, 1000]
    pool = _filled(gen, lens, hkv, bs, table, shift=1.0)
    q = (torch.randn(len(lens), hkv * G, 192, generator=gen, device=DEV) * 1.5).bfloat16()
    pos = [n - 1 for n in lens]
    seq = list(range(len(lens)))
    out = kvr.full_attn_decode_kv4(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, 1000)
    assert kvr.device_status() == 0
    _check_decode(out, q, pos, seq, pool, table)


@pytest.mark.parametrize("ctx,hkv,G,dist", [(8193, 1, 16, 0.0), (20001, 2, 16, 3.0), (65537, 1, 8, 1.0)])
def test_decode_long(table, ctx, hkv, G, dist):
    gen = _gen(ctx)
    pool = _filled(gen, [ctx], hkv, 64, table, shift=dist)
    q = (torch.randn(2, hkv * G, 192, generator=gen, device=DEV) * 2).bfloat16()
    pos = [ctx - 1, ctx // 2]
    out = kvr.full_attn_decode_kv4(q, _ints(pos, torch.int64), _ints([0, 0], torch.int32), pool, table, SCALE, ctx)
    _check_decode(out, q, pos, [0, 0], pool, table)
    assert kvr.device_status() == 0


def test_decode_draft_rows_share_a_sequence(table):
    gen = _gen(31)
    lens, C, hkv, G = [70, 300, 1025], 4, 2, 8
    pool = _filled(gen, lens, hkv, 32, table)
    pos = [n - C + c for n in lens for c in range(C)]
    seq = [s for s in range(len(lens)) for _ in range(C)]
    q = torch.randn(len(pos), hkv * G, 192, generator=gen, device=DEV).bfloat16()
    out = kvr.full_attn_decode_kv4(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, 1025)
    _check_decode(out, q, pos, seq, pool, table)


@pytest.mark.parametrize("vscales", [(1e-6,), (2e4,), (1.0, 1e-5, 3e3, 1e-2), (1e-3, 6e4)])
def test_decode_value_scales_apart(table, vscales):
    """Values whose scales differ by orders of magnitude from token to token, in both orders of appearance."""
    gen = _gen(41)
    n, hkv, G = 600, 1, 16
    for flip in (False, True):
        pool = _pool(gen, 1, hkv, n, 64)
        k, v = _kv(gen, n, hkv)
        f = torch.tensor(vscales, device=DEV).repeat(n // len(vscales) + 1)[:n].sort(descending=flip).values
        _append(pool, k, (v.float() * f[:, None, None]).bfloat16(), 0, 0, table)
        q = torch.randn(1, G, 192, generator=gen, device=DEV).bfloat16()
        out = kvr.full_attn_decode_kv4(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
        _check_decode(out, q, [n - 1], [0], pool, table, f"{vscales} {flip}")


@pytest.mark.parametrize("mag", [0.0, 1e-30, 1e-3, 30.0, 1e4])
def test_decode_query_magnitudes(table, mag):
    """Queries of any size: zeros (all keys weigh the same), tiny, and so large that one key takes everything."""
    gen = _gen(43)
    n, hkv, G = 200, 2, 4
    pool = _filled(gen, [n], hkv, 64, table)
    q = (torch.randn(1, hkv * G, 192, generator=gen, device=DEV) * mag).bfloat16()
    out = kvr.full_attn_decode_kv4(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
    if mag < 1e3:
        _check_decode(out, q, [n - 1], [0], pool, table)
    else:  # the weights are one key's or split by rounding between near ties: the value of a key that is near the best
        K, V, ok = o4.sequence(pool.data.cpu().numpy(), pool.block_table[0].cpu().numpy(), 0, n)
        assert torch.isfinite(out).all()
        assert float(out.abs().max()) <= np.abs(V).max() * 1.01 or hkv > 1


def test_decode_scores_rise_and_fall(table):
    """Scores that climb along the keys (every tile raises the maximum) and that fall by hundreds (late keys weigh
    nothing), and one far above the rest at either end."""
    gen = _gen(47)
    n, G = 1500, 16
    u = torch.zeros(192, device=DEV)
    u[64:] = torch.randn(128, generator=gen, device=DEV)
    u /= u.norm()
    for ramp in (torch.linspace(-300, 300, n), torch.linspace(300, -300, n), torch.eye(n)[0] * 400, torch.eye(n)[-1] * 400):
        pool = _pool(gen, 1, 1, n, 64)
        k, v = _kv(gen, n, 1)
        k = (k.float() * 0.05 + ramp.to(DEV)[:, None, None] * u * 0.5).bfloat16()
        _append(pool, k, v, 0, 0, table)
        q = (torch.randn(1, G, 192, generator=gen, device=DEV) * 0.1 + u * 14).bfloat16()
        out = kvr.full_attn_decode_kv4(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
        # scores of hundreds carry the fp16 rounding of q: 2^-10 of sum |q||k| is up to 0.6, so the bound of
        # _check_decode is wide here (the weights' change taken as the exponential it is, of values that differ by at
        # most 2 |v|_max), and the rel RMS bar does not apply: check the bound alone
        K, V, ok = o4.sequence(pool.data.cpu().numpy(), pool.block_table[0].cpu().numpy(), 0, n)
        want, a, w = o4.attend(q[0].float().cpu().numpy(), n - 1, K, V, ok, table[n - 1].cpu().numpy(), SCALE)
        err = np.abs(out[0].double().cpu().numpy() - want)
        tol = 2.0 ** -8 * np.abs(want) + (np.exp(2 * 2.0 ** -10 * a[:, None]) - 1) * 2 * np.abs(V).max() + 2.0 ** -10 * (w + 3 * np.abs(V).max())
        assert np.all(err <= tol)


def test_decode_nan_and_what_lies_behind(table):
    gen = _gen(53)
    n, hkv, G = 100, 2, 4
    pool = _filled(gen, [n, n], hkv, 16, table)   # 0xFF (NaN scales) wherever nothing was written
    k, v = _kv(gen, 1, hkv)
    v[0, 1, 70] = float("nan")                    # value group 1 of KV head 1 of the last key of sequence 0
    _append(pool, k, v, 0, n - 1, table)
    k2 = k.clone()
    k2[0, 0, 0] = float("inf")                    # a key of KV head 0 of sequence 1
    _append(pool, k2, _kv(gen, 1, hkv)[1], 1, 40, table)
    q = torch.randn(2, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pos, seq = _ints([n - 1, n - 1], torch.int64), _ints([0, 1], torch.int32)
    out = kvr.full_attn_decode_kv4(q, pos, seq, pool, table, SCALE, n)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[0, G:, 64:] = True
    want[1, :G] = True
    assert torch.equal(nan, want)
    # a query before the bad key does not see it
    out = kvr.full_attn_decode_kv4(q, _ints([n - 2, 39], torch.int64), seq, pool, table, SCALE, n)
    assert torch.isfinite(out).all()
    # a query holding a NaN or an infinity spoils its own head only
    q[0, 1, 3] = float("nan")
    q[0, 2, 100] = float("inf")
    out = kvr.full_attn_decode_kv4(q, _ints([n - 2, 39], torch.int64), seq, pool, table, SCALE, n)
    bad = torch.zeros_like(nan)
    bad[0, 1:3] = True
    assert torch.equal(torch.isnan(out), bad)


def test_decode_bad_rows_and_blocks(table):
    gen = _gen(59)
    n, hkv, G = 200, 2, 8
    pool = _filled(gen, [n] * 5, hkv, 32, table)
    pool.block_table[1, 2] = -1
    pool.block_table[2, 0] = pool.num_blocks
    pool.block_table[4, :] = -7
    q = torch.randn(7, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    seq = [0, 1, 2, 9, -1, 3, 4]
    pos = [n - 1, n - 1, n - 1, 5, 5, n, n - 1]
    out = kvr.full_attn_decode_kv4(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, n,
                                   out=torch.full((7, hkv * G, 128), 7.0, dtype=torch.bfloat16, device=DEV))
    assert kvr.device_status() == kvr.DEV_BAD_POS | kvr.DEV_BAD_SEQ | kvr.DEV_BAD_BLOCK
    for b in (3, 4, 5, 6):
        assert not out[b].any(), b
    _check_decode(out[:3], q[:3], pos[:3], seq[:3], pool, table)  # bad blocks' keys count as masked


def test_decode_repeats_bit_for_bit_and_in_graphs(table):
    gen = _gen(61)
    lens, hkv, G = [3000, 17, 800], 4, 16
    pool = _filled(gen, lens, hkv, 64, table, max_ctx=4096)
    q = torch.randn(3, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pos, seq = _ints([n - 1 for n in lens], torch.int64), _ints([0, 1, 2], torch.int32)
    first = kvr.full_attn_decode_kv4(q, pos, seq, pool, table, SCALE, 4096)
    for _ in range(5):
        assert torch.equal(kvr.full_attn_decode_kv4(q, pos, seq, pool, table, SCALE, 4096), first)
    # two captured graphs on two streams, each with a workspace of its own, replayed side by side with other lengths
    n = kvr.full_attn_decode_kv4_workspace_size(3, hkv * G, hkv, 4096)
    runs = []
    for i in range(2):
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        p, out = pos.clone(), torch.empty_like(first)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            kvr.full_attn_decode_kv4(q, p, seq, pool, table, SCALE, 4096, workspace=ws, out=out)
        runs.append((g, p, out, st, ws))
    torch.cuda.synchronize()
    runs[1][1].copy_(_ints([40, 3, 799], torch.int64))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, _, _, st, _ in runs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(runs[0][2], first)
    _check_decode(runs[1][2], q, [40, 3, 799], [0, 1, 2], pool, table)


@pytest.mark.parametrize("B", [3, 128, 150, 300])
def test_decode_of_positions_written_right_before(table, B):
    """Positions and ids come from the kernel launched just ahead, other ones each time: what a decode reads of the batch
    before that kernel is done never counts."""
    gen = _gen(70 + B)
    hkv, G, ctx, bs = 2, 16, 4096, 64
    pool = _filled(gen, [ctx, ctx, ctx], hkv, bs, table, max_ctx=ctx)
    pool = kvr.Kv4Layout(pool.data, pool.block_table[torch.arange(B, device=DEV) % 3].contiguous())
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    own = torch.zeros(B, ctx // bs, dtype=torch.int32, device=DEV)
    free, left = torch.zeros(B, dtype=torch.int32, device=DEV), _ints([B], torch.int32)
    cu, count = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    pos, slots = torch.zeros(B, dtype=torch.int64, device=DEV), torch.empty(B, dtype=torch.int64, device=DEV)
    seq, add = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    ws = torch.empty(kvr.full_attn_decode_kv4_workspace_size(B, hkv * G, hkv, ctx), dtype=torch.uint8, device=DEV)
    steps = []
    for _ in range(12):
        lens = torch.randint(0, 200, (B,), generator=gen, device=DEV)
        lens[torch.randint(0, B, (2,), generator=gen, device=DEV)] = torch.randint(0, ctx, (2,), generator=gen, device=DEV)
        steps.append((lens, torch.randperm(B, generator=gen, device=DEV).to(torch.int32),
                      torch.empty(B, hkv * G, 128, dtype=torch.bfloat16, device=DEV)))
    torch.cuda.synchronize()
    for lens, ids, out in steps:
        kvr.kv_pages_grow(own, 1, bs, ids, lens, add, free, left, cu, pos, seq, slots, free_count_out=count)
        kvr.full_attn_decode_kv4(q, pos, seq, pool, table, SCALE, ctx, workspace=ws, out=out)
    torch.cuda.synchronize()
    for lens, ids, out in steps:
        assert torch.equal(out, kvr.full_attn_decode_kv4(q, lens, ids, pool, table, SCALE, ctx))
    assert kvr.device_status() == 0
    lens, ids, out = steps[-1]
    few = [0, 1, 2] if B > 3 else list(range(B))
    _check_decode(out[few], q[few], lens[few].tolist(), ids[few].tolist(), pool, table)


@pytest.mark.parametrize("B", [33, 130, 700])
def test_decode_many_sequences(table, B):
    gen = _gen(B)
    hkv, G = 1, 2
    lens = torch.randint(1, 90, (B,), generator=gen, device=DEV).tolist()
    pool = _pool(gen, B, hkv, 90, 16)
    n = sum(lens)
    k, v = _kv(gen, n, hkv)
    seq = torch.arange(B, device=DEV).repeat_interleave(torch.tensor(lens, device=DEV)).to(torch.int32)
    pos = torch.cat([torch.arange(m, device=DEV) for m in lens])
    kvr.kv4_append_rope(k, v, pos, seq, table, VS, pool)
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    last = [m - 1 for m in lens]
    out = kvr.full_attn_decode_kv4(q, _ints(last, torch.int64), torch.arange(B, device=DEV).to(torch.int32), pool, table,
                                   SCALE, 90)
    _check_decode(out, q, last, list(range(B)), pool, table)


# -- unpack --------------------------------------------------------------------------------------------------------------

def _bf16(x):
    """fp64 -> fp32 -> bf16, round to nearest even twice, as the kernel's sum and store."""
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def _want_unpacked(pool, s, lo, n):
    data, bt = pool.data.cpu().numpy(), pool.block_table.cpu().numpy()
    ks, vs = [], []
    for h in range(pool.num_kv_heads):
        K, V, ok = o4.sequence(data, bt[s], h, lo + n)
        K[~ok], V[~ok] = 0, 0
        ks.append(_bf16(K[lo:]))
        vs.append(_bf16(V[lo:]))
    return torch.stack(ks, 1), torch.stack(vs, 1)


@pytest.mark.parametrize("bs,dbs", [(16, 16), (48, 64), (64, 32), (256, 16)])
@pytest.mark.parametrize("kind", ["linear", "paged"])
def test_unpack(table, kind, bs, dbs):
    gen = _gen(bs + dbs)
    lens, hkv = [400, 33, 700, 90], 3
    pool = _filled(gen, lens, hkv, bs, table, shift=1.0)
    seqs = [2, 0, 1, 2, 3, 3]
    lo = [5, 399, 0, 0, 16, 20]
    rows = [333, 1, 33, 0, 47, 3] if kind == "linear" else [333, 1, 33, 0, 4, 3]
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    args = (_ints(seqs, torch.int32), _ints(lo, torch.int64), _ints(cu, torch.int32))
    if kind == "linear":
        dst = kvr.LinearLayout.empty(cu[-1] + 9, hkv)
        dst.k.fill_(9)
        dst.v.fill_(9)
        kvr.kv4_unpack(pool, *args, dst)
        for i, (s, a, n) in enumerate(zip(seqs, lo, rows)):
            if n:
                k, v = _want_unpacked(pool, s, a, n)
                assert torch.equal(dst.k[cu[i]:cu[i + 1]].cpu(), k) and torch.equal(dst.v[cu[i]:cu[i + 1]].cpu(), v), i
        assert (dst.k[cu[-1]:] == 9).all() and (dst.v[cu[-1]:] == 9).all()  # rows past the last entry stay
    else:
        dst = kvr.PagedLayout.contiguous(7, hkv, 704, block_size=dbs)
        dst.k.fill_(9)
        dst.v.fill_(9)
        dseq = [4, 0, 1, 2, 3, 6]
        kvr.kv4_unpack(pool, *args, dst, dst_seqs=_ints(dseq, torch.int32), T=cu[-1])
        left = torch.ones(7, dst.max_blocks * dbs, dtype=torch.bool)
        kk = dst.k.view(7, dst.max_blocks, hkv, dbs, 192).transpose(2, 3).reshape(7, -1, hkv, 192).cpu()
        vv = dst.v.view(7, dst.max_blocks, hkv, dbs, 128).transpose(2, 3).reshape(7, -1, hkv, 128).cpu()
        for s, d, a, n in zip(seqs, dseq, lo, rows):
            if n:
                k, v = _want_unpacked(pool, s, a, n)
                assert torch.equal(kk[d, a:a + n], k) and torch.equal(vv[d, a:a + n], v)
                left[d, a:a + n] = False
        assert (kk[left] == 9).all() and (vv[left] == 9).all()              # and so do the other positions
    assert kvr.device_status() == 0


def test_unpack_flags(table):
    gen = _gen(71)
    hkv = 2
    pool = _filled(gen, [100, 100], hkv, 32, table)
    pool.block_table[1, 1] = -1
    cu = [0, 50, 60, 70, 80, 90]
    dst = kvr.LinearLayout.empty(100, hkv)
    dst.k.fill_(9)
    kvr.kv4_unpack(pool, _ints([1, 2, -1, 0, 0], torch.int32), _ints([10, 0, 0, -5, 1 << 50], torch.int64),
                   _ints(cu, torch.int32), dst)
    assert kvr.device_status() == kvr.DEV_BAD_BLOCK | kvr.DEV_BAD_SEQ | kvr.DEV_BAD_POS
    k, _ = _want_unpacked(pool, 1, 10, 50)
    assert not k[22:].any() and torch.equal(dst.k[:50].cpu(), k)
    assert not dst.k[50:90].any() and (dst.k[90:] == 9).all()
    # row ranges that leave the call
    dst.k.fill_(9)
    kvr.kv4_unpack(pool, _ints([0], torch.int32), _ints([0], torch.int64), _ints([40, 30], torch.int32), dst)
    assert kvr.device_status() == kvr.DEV_BAD_ROWS
    kvr.kv4_unpack(pool, _ints([0], torch.int32), _ints([0], torch.int64), _ints([90, 101], torch.int32), dst)
    assert kvr.device_status() == kvr.DEV_BAD_ROWS
    kvr.kv4_unpack(pool, _ints([0], torch.int32), _ints([0], torch.int64), _ints([-1, 30], torch.int32), dst)
    assert kvr.device_status() == kvr.DEV_BAD_ROWS
    assert (dst.k == 9).all()
    # pages that cannot be addressed
    pages = kvr.PagedLayout.contiguous(2, hkv, 64, block_size=32)
    pages.k.fill_(9)
    pages.block_table[0, 1] = pages.num_blocks
    kvr.kv4_unpack(pool, _ints([0, 0], torch.int32), _ints([0, 0], torch.int64), _ints([0, 64, 90], torch.int32), pages,
                   dst_seqs=_ints([0, 2], torch.int32))
    assert kvr.device_status() == kvr.DEV_BAD_BLOCK | kvr.DEV_BAD_SEQ
    assert torch.equal(pages.k[0].transpose(0, 1).cpu(), _want_unpacked(pool, 0, 0, 32)[0]) and (pages.k[1:] == 9).all()


# -- page growth ---------------------------------------------------------------------------------------------------------

def _grow(tab, bs, nb, seqs, lens, add, free, count, T, in_place=True):
    n = len(seqs)
    t = _ints(tab.tolist(), torch.int32)
    ids, cnt = _ints(free.tolist(), torch.int32), _ints([count], torch.int32)
    left = None if in_place else torch.full((1,), -99, dtype=torch.int32, device=DEV)
    cu = torch.full((n + 1,), 77, dtype=torch.int32, device=DEV)
    pos, rs, sl = (torch.full((T,), 77, dtype=d, device=DEV) for d in (torch.int64, torch.int32, torch.int64))
    kvr.kv_pages_grow(t, nb, bs, _ints(list(seqs), torch.int32), _ints(list(lens), torch.int64),
                      _ints(list(add), torch.int32), ids, cnt, cu, pos, rs, sl, free_count_out=left)
    if not in_place:
        assert int(cnt) == count
    assert torch.equal(ids.cpu(), torch.from_numpy(free))
    flags = kvr.device_status()
    want = o4.grow(tab, bs, nb, seqs, lens, add, free, count, T)
    got = (t, cnt if in_place else left, cu, pos, rs, sl)
    for name, a, b in zip(("table", "count", "cu_rows", "pos", "row_seq", "slots"), got, want):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1)), name
    assert flags == want[6]
    return flags


def _state(rng, S, mb, bs, seqs, lens):
    nb = S * mb + 5
    ids = rng.permutation(nb).astype(np.int32)
    tab = np.full((S, mb), -1, np.int32)
    at = 0
    for s, n in zip(seqs, lens):
        held = -(-n // bs)
        tab[s, :held] = ids[at:at + held]
        at += held
    free = np.full(nb, -1, np.int32)
    free[:nb - at] = ids[at:]
    return tab, nb, free, nb - at


@pytest.mark.parametrize("n,bs,most,S,mb", [(1, 16, 1, 1, 4), (3, 16, 40, 5, 8), (64, 64, 1, 64, 16), (100, 48, 200, 130, 12),
                                            (1025, 16, 60, 1100, 9), (8192, 64, 3, 8192, 4)])
def test_grow(n, bs, most, S, mb):
    rng = np.random.default_rng(n + bs)
    seqs = rng.permutation(S)[:n].astype(np.int32)
    lens = rng.integers(0, mb * bs - most + 1, n)
    lens[rng.random(n) < 0.3] //= bs
    lens[rng.random(n) < 0.3] //= bs
    lens = np.where(rng.random(n) < 0.3, lens // bs * bs, lens)
    add = np.where(rng.random(n) < 0.3, 0, rng.integers(0, most + 1, n))
    tab, nb, free, count = _state(rng, S, mb, bs, seqs, lens)
    T = int(add.sum())
    for pad, in_place in ((0, True), (9000, False)):
        assert _grow(tab, bs, nb, seqs, lens, add, free, count, T + pad, in_place) == 0


def test_grow_flags():
    rng = np.random.default_rng(5)
    S, mb, bs = 6, 4, 16
    seqs, lens, add = [0, 1, 2, 3], [10, 0, 16, 63], [7, 33, 0, 1]
    tab, nb, free, count = _state(rng, S, mb, bs, seqs, lens)
    call = lambda **kw: _grow(**{**dict(tab=tab, bs=bs, nb=nb, seqs=seqs, lens=lens, add=add, free=free, count=count, T=50), **kw})
    assert call() == 0
    need = 4
    assert call(count=need, free=free[:need].copy()) == 0                    # the last block
    assert call(count=need - 1) == kvr.DEV_NO_BLOCKS and call(count=0) == kvr.DEV_NO_BLOCKS
    assert call(count=-1) == kvr.DEV_NO_BLOCKS and call(count=len(free) + 1) == kvr.DEV_NO_BLOCKS
    assert call(T=41) == 0 and call(T=40) == kvr.DEV_BAD_ROWS and call(T=0) == kvr.DEV_BAD_ROWS
    assert call(seqs=[0, 6, -1, 3]) == kvr.DEV_BAD_SEQ
    assert call(lens=[10, -1, 16, 2 ** 62], add=[7, 33, 0, 1]) == kvr.DEV_BAD_POS
    assert call(add=[7, -3, 0, 2]) == kvr.DEV_BAD_POS
    assert call(add=[7, 2 ** 31 - 1, 0, 2 ** 31 - 1]) == kvr.DEV_BAD_POS
    wide = np.full((6, 2 ** 12), -1, np.int32)                               # row sums past 31 bits
    assert _grow(wide, 2 ** 20, 4, seqs, [0] * 4, [2 ** 31 - 1] * 4, free, count, 10) == kvr.DEV_BAD_ROWS
    bad = free.copy()
    bad[count - 1], bad[count - 2] = nb, -4                                  # ids that are none of the pool's
    assert call(free=bad) == kvr.DEV_BAD_BLOCK
    hole = tab.copy()
    hole[0, 0] = -1                                                          # a block that should be held already
    assert call(tab=hole) == kvr.DEV_BAD_BLOCK
    assert call(seqs=[], lens=[], add=[]) == 0


# -- together ------------------------------------------------------------------------------------------------------------

def test_a_run_of_them_together(table):
    """Three requests served for some steps: grow makes the step's rows, the append takes its slot map, single tokens
    decode over the 4-bit pool, chunks go through unpacked pages and the varlen prefill, and a finished request's blocks
    go back to the free list that the next one's come from.  The append and decode run inside one captured graph."""
    gen = _gen(97)
    hkv, G, bs, S, mb = 2, 8, 32, 4, 12
    nb, T = 20, 150
    data = torch.full((nb, hkv, bs // 16, kvr.KV4_TILE), 0xFF, dtype=torch.uint8, device=DEV)
    bt = torch.full((S, mb), -1, dtype=torch.int32, device=DEV)
    pool = kvr.Kv4Layout(data, bt)
    free = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    count = _ints([nb], torch.int32)
    n = 3
    seqs = _ints([2, 0, 3], torch.int32)
    lens, add = torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    cu = torch.empty(n + 1, dtype=torch.int32, device=DEV)
    pos, rs, sl = (torch.empty(T, dtype=d, device=DEV) for d in (torch.int64, torch.int32, torch.int64))
    k = torch.zeros(T, hkv, 192, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(T, hkv, 128, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(T, hkv * G, 192, dtype=torch.bfloat16, device=DEV)
    qd, outd = torch.zeros(n, hkv * G, 192, dtype=torch.bfloat16, device=DEV), torch.zeros(n, hkv * G, 128, dtype=torch.bfloat16, device=DEV)
    last = torch.zeros(n, dtype=torch.int64, device=DEV)
    ws = torch.empty(kvr.full_attn_decode_kv4_workspace_size(n, hkv * G, hkv, mb * bs), dtype=torch.uint8, device=DEV)

    def step():
        kvr.kv_pages_grow(bt, nb, bs, seqs, lens, add, free, count, cu, pos, rs, sl)
        kvr.kv4_append_rope(k, v, pos, None, table, VS, pool, slots=sl)
        kvr.full_attn_decode_kv4(qd, last, seqs, pool, table, SCALE, mb * bs, workspace=ws, out=outd)

    step()  # an empty step first: nothing is added, the decode reads position 0 of empty tables
    kvr.device_status(reset=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step()
    pages = kvr.PagedLayout.contiguous(n, hkv, mb * bs, block_size=64)
    ids3 = _ints([0, 1, 2], torch.int32)
    held = [0, 0, 0]
    for adds in ([100, 7, 33], [1, 1, 1], [1, 40, 1], [4, 1, 90], [1, 1, 1]):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        add.copy_(_ints(adds, torch.int32))
        lens.copy_(_ints(held, torch.int64))
        last.copy_(lens + add - 1)
        cur = np.concatenate([[0], np.cumsum(adds)])
        qd.copy_(q[torch.from_numpy(cur[1:] - 1).to(DEV)])
        g.replay()
        torch.cuda.synchronize()
        assert kvr.device_status() == 0
        held = [a + b for a, b in zip(held, adds)]
        assert int(count) == nb - sum(-(-h // bs) for h in held)
        assert cu.tolist() == cur.tolist()
        _check_decode(outd, qd, [h - 1 for h in held], seqs.tolist(), pool, table)
        # the same rows through bf16 pages and the varlen call
        hold = _ints(np.concatenate([[0], np.cumsum(held)]).tolist(), torch.int32)
        kvr.kv4_unpack(pool, seqs, torch.zeros(n, dtype=torch.int64, device=DEV), hold, pages, dst_seqs=ids3, T=sum(held))
        rows = int(cur[-1])
        out = kvr.full_attn_prefill_varlen(q[:rows].contiguous(), cu, lens, ids3, pages, table, SCALE, mb * bs)
        ends = out[torch.from_numpy(cur[1:] - 1).to(DEV)].float()
        # both round to bf16 (half a step each) and the varlen path's q, values and weights too: 2^-6 in all, of |v| < 4
        assert float((ends - outd.float()).abs().max()) <= 4 * 2.0 ** -6
        # every row of the batch as a decode row of its own
        own = kvr.full_attn_decode_kv4(q[:rows].contiguous(), pos[:rows].contiguous(), rs[:rows].contiguous(), pool, table,
                                       SCALE, mb * bs)
        assert float((own.float() - out.float()).abs().max()) <= 4 * 2.0 ** -6
        assert torch.equal(own[torch.from_numpy(cur[1:] - 1).to(DEV)], outd) or rows != n
    # request 0 ends: its blocks go back, and a new one in its place takes them
    kvr.kv_pages_release_window(bt, nb, bs, seqs[:1].contiguous(), _ints([mb * bs], torch.int64), free, count, window=1)
    assert int(count) == nb - sum(-(-h // bs) for h in held[1:]) and (bt[2] == -1).all()
    assert kvr.device_status() == 0


@pytest.mark.parametrize("by_slot", [False, True])
@pytest.mark.parametrize("bs", [16, 48, 64])
def test_append_runs(table, bs, by_slot):
    """Runs of every kind in one call: whole tiles at every offset of the call, chunks that start and end inside a tile,
    runs cut by padding, backwards and repeated order, neighbours in memory that are not neighbours in a sequence."""
    gen = _gen(300 + bs)
    hkv, S = 2, 8
    pool = _pool(gen, S, hkv, 1024, bs, fill=0xEE)
    runs = [(0, 0, 16), (1, 5, 11), (1, 16, 16), (1, 32, 37), (2, 3, 1), (0, 16, 100), (3, 1, 15), (4, 15, 1), (4, 16, 17),
            (5, 500, 33), (None, 0, 7), (5, 533, 11), (6, 0, 15), (None, 0, 1), (6, 15, 1), (6, 16, 16), (7, 64, 64),
            (2, 128, 64), (0, 116, 12), (3, 16, 16), (3, 32, 3)]
    seq, pos = [], []
    for s, lo, n in runs:
        seq += [-1 if s is None else s] * n
        pos += [-1] * n if s is None else list(range(lo, lo + n))
    back = list(range(700, 732))[::-1]
    seq += [7] * 32
    pos += back
    T = len(seq)
    k, v = _kv(gen, T, hkv, 1.0)
    seq_t, pos_t = _ints(seq, torch.int32), _ints(pos, torch.int64)
    bt = pool.block_table.cpu().numpy()
    places = [None if s < 0 else (int(bt[s, p // bs]), p % bs) for s, p in zip(seq, pos)]
    want = _want_bytes(pool, k, v, places, pos_t, table)
    if by_slot:
        slots = _ints([-1 if pl is None else pl[0] * bs + pl[1] for pl in places], torch.int64)
        kvr.kv4_append_rope(k, v, pos_t, None, table, VS, pool, slots=slots)
    else:
        kvr.kv4_append_rope(k, v, pos_t, seq_t, table, VS, pool)
    assert np.array_equal(pool.data.cpu().numpy(), want)
    assert kvr.device_status() == 0


def test_decode_long_shares_keep_their_digits(table):
    """Long shares per CTA (18,000 keys): the codes' sums (all positive) and the minima's cancel to a hundredth of their
    size, so a sum cut off below its last bit at every product would show.  The output's own rounding is at most 2^-8 of
    a value, 2^-8 / sqrt(3) in the mean square; everything else (weights and scaled weights rounded to fp16, 2^-11 each
    and independent from key to key) is held to 2^-11."""
    gen = _gen(211)
    B, ctx, hkv, G = 32, 65537, 4, 16
    pool = kvr.Kv4Layout.contiguous(B, hkv, ctx, zero=False)
    for s in range(B):
        _append(pool, *_kv(gen, ctx, hkv, 0.5), s, 0, table)
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pos = torch.full((B,), ctx - 1, dtype=torch.int64, device=DEV)
    out = kvr.full_attn_decode_kv4(q, pos, torch.arange(B, dtype=torch.int32, device=DEV), pool, table, SCALE, ctx)
    pl = [o4.places(r) for r in range(16)]
    at = [torch.tensor(np.array([p[i] for p in pl]), device=DEV) for i in range(6)]
    hi = (torch.arange(192, device=DEV) % 2 * 4).to(torch.uint8)

    def group(tiles, codes, scales, minima, n):
        half = lambda a: torch.stack([tiles[:, a], tiles[:, a + 1]], -1).contiguous().view(torch.float16)[..., 0].double()
        u = ((tiles[:, codes] >> hi[:n]) & 15).double()
        return (half(minima).repeat_interleave(64, -1) + half(scales).repeat_interleave(64, -1) * u).flatten(0, 1)

    cs = table[ctx - 1].double()
    for b, h in ((0, 0), (17, 3), (31, 1)):
        tiles = pool.data[pool.block_table[b].long(), h].flatten(0, 1)
        K, V = group(tiles, at[0], at[2], at[5], 192)[:ctx], group(tiles, at[1], at[3], at[4], 128)[:ctx]
        x = q[b, h * G:(h + 1) * G].double()
        x = torch.cat([x[:, :32] * cs[:, 0] - x[:, 32:64] * cs[:, 1], x[:, 32:64] * cs[:, 0] + x[:, :32] * cs[:, 1], x[:, 64:]], 1)
        want = torch.softmax(x @ K.T * SCALE, -1) @ V
        err = (out[b, h * G:(h + 1) * G].double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(err.max()) <= 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -11, float(err.max())


@pytest.mark.parametrize("G", [3, 8, 16])
def test_decode_ragged_rows_share_ctas(table, G):
    """Many short and some long rows, several to a CTA, rows cut at a CTA's share: bit for bit the same in every run, and
    right in a sample of rows of every length."""
    gen = _gen(307 + G)
    B, hkv, most = 150, 4, 6000
    lens = torch.exp(torch.rand(B, generator=gen, device=DEV) * np.log(most)).long().clamp(1, most).tolist()
    pool = _pool(gen, B, hkv, most, 48)
    k, v = _kv(gen, sum(lens), hkv, 1.0)
    seq = torch.arange(B, device=DEV).repeat_interleave(torch.tensor(lens, device=DEV)).to(torch.int32)
    kvr.kv4_append_rope(k, v, torch.cat([torch.arange(m, device=DEV) for m in lens]), seq, table, VS, pool)
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pos, ids = _ints([m - 1 for m in lens], torch.int64), torch.arange(B, dtype=torch.int32, device=DEV)
    n = kvr.full_attn_decode_kv4_workspace_size(B, hkv * G, hkv, most)
    outs = []
    for i in range(12):
        ws = torch.full((n,), 0xFF if i % 2 else 0, dtype=torch.uint8, device=DEV)  # no initialisation is relied on
        outs.append(kvr.full_attn_decode_kv4(q, pos, ids, pool, table, SCALE, most, workspace=ws))
    assert all(torch.equal(o, outs[0]) for o in outs)
    some = sorted(range(B), key=lambda b: lens[b])[::5]
    _check_decode(outs[0][some], q[some], [lens[b] - 1 for b in some], some, pool, table)


@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("B,hkv,max_ctx", [(1, 1, 1), (1, 2, 2048), (9, 1, 2048), (14, 4, 2049), (50, 4, 1024), (120, 8, 1000),
                                           (300, 2, 64)])
def test_decode_short_contexts(table, G, B, hkv, max_ctx):
    """Batches around the sizes where a row is taken by a cluster of CTAs in one launch: contexts from one token to the
    bound, rows that cannot be served among them, a captured run replayed with other lengths."""
    gen = _gen(401 + B + G)
    lens = torch.randint(1, max_ctx + 1, (B,), generator=gen, device=DEV).tolist()
    lens[0] = max_ctx
    if B > 3:
        lens[1], lens[2] = 1, min(33, max_ctx)
    pool = _pool(gen, B, hkv, max_ctx, 32)
    k, v = _kv(gen, sum(lens), hkv, 1.0)
    seq = torch.arange(B, device=DEV).repeat_interleave(torch.tensor(lens, device=DEV)).to(torch.int32)
    kvr.kv4_append_rope(k, v, torch.cat([torch.arange(m, device=DEV) for m in lens]), seq, table, VS, pool)
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pos, ids = _ints([m - 1 for m in lens], torch.int64), torch.arange(B, dtype=torch.int32, device=DEV)
    bad = 3 if B > 3 else None
    if bad is not None:
        pos[bad] = max_ctx
    out = torch.full((B, hkv * G, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(kvr.full_attn_decode_kv4_workspace_size(B, hkv * G, hkv, max_ctx), dtype=torch.uint8, device=DEV)
    call = lambda: kvr.full_attn_decode_kv4(q, pos, ids, pool, table, SCALE, max_ctx, workspace=ws, out=out)
    call()
    assert kvr.device_status() == (kvr.DEV_BAD_POS if bad is not None else 0)
    good = [b for b in range(B) if b != bad]
    some = good if B <= 20 else good[::7] + [0, 1, 2]
    if bad is not None:
        assert not out[bad].any()
    _check_decode(out[some], q[some], [lens[b] - 1 for b in some], some, pool, table)
    first = out.clone()
    call()
    assert torch.equal(out, first)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    half = [max(1, m // 2) for m in lens]
    pos.copy_(_ints([m - 1 for m in half], torch.int64))
    g.replay()
    torch.cuda.synchronize()
    kvr.device_status()
    _check_decode(out[some], q[some], [half[b] - 1 for b in some], some, pool, table)


def test_unpack_rows_at_any_aligned_address(table):
    """Destinations whose rows start 16 but not 32 bytes on (the store width goes by it)."""
    gen = _gen(73)
    hkv, n = 2, 70
    pool = _filled(gen, [n], hkv, 16, table)
    args = (_ints([0], torch.int32), _ints([0], torch.int64), _ints([0, n], torch.int32))
    want = _want_unpacked(pool, 0, 0, n)
    for shift in (0, 8):
        kb = torch.full((n * hkv * 192 + 64,), 9.0, dtype=torch.bfloat16, device=DEV)
        vb = torch.full((n * hkv * 128 + 64,), 9.0, dtype=torch.bfloat16, device=DEV)
        k = kb[shift:shift + n * hkv * 192].view(n, hkv, 192)
        v = vb[shift:shift + n * hkv * 128].view(n, hkv, 128)
        kvr.kv4_unpack(pool, *args, kvr.LinearLayout(k, v))
        assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
        assert (kb[shift + k.numel():] == 9).all() and (kb[:shift] == 9).all()


@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("ctx", [700, 20000])
def test_decode_stalled_wait_leaves_in_time(table, ctx, G):
    """A wait that nothing completes runs into its limit: the kernel leaves with the timeout bit (the cluster form for the
    short context, the work line for the long one), and the next call is right again."""
    gen = _gen(503 + ctx + G)
    pool = _filled(gen, [ctx, 40], 2, 64, table)
    q = torch.randn(2, 2 * G, 192, generator=gen, device=DEV).bfloat16()
    pos, ids = _ints([ctx - 1, 39], torch.int64), _ints([0, 1], torch.int32)
    call = lambda: kvr.full_attn_decode_kv4(q, pos, ids, pool, table, SCALE, ctx)
    want = call()
    assert kvr.device_status() == 0
    kvr.debug_stall_next(1, 2_000_000)
    call()
    assert kvr.device_status() & kvr.DEV_TIMEOUT
    assert torch.equal(call(), want)
    assert kvr.device_status() == 0
    kvr.debug_stall_next(0, 1000)


def test_decode_on_another_stream(table):
    gen = _gen(509)
    pool = _filled(gen, [900, 3000], 2, 64, table)
    q = torch.randn(2, 16, 192, generator=gen, device=DEV).bfloat16()
    pos, ids = _ints([899, 2999], torch.int64), _ints([0, 1], torch.int32)
    want = kvr.full_attn_decode_kv4(q, pos, ids, pool, table, SCALE, 3000)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    outs = [kvr.full_attn_decode_kv4(q, pos, ids, pool, table, SCALE, 3000, stream=st) for _ in range(20)]
    junk = [torch.randn(1 << 20, device=DEV) for _ in range(20)]  # the current stream goes on allocating meanwhile
    st.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and len(junk) == 20


def test_pools_past_4_gb(table):
    """Blocks whose bytes lie past 32 bits, in the 4-bit pool and in the bf16 pages they are unpacked to, give what a
    pool of three blocks gives."""
    gen = _gen(95)
    n, bs, G, nb = 2100, 1024, 16, 24000                                    # 4.5 GB of tiles
    k, v = _kv(gen, n, 1)
    q = torch.randn(2, G, 192, generator=gen, device=DEV).bfloat16()
    pos, seq = _ints([n - 1, 1500], torch.int64), _ints([0, 0], torch.int32)
    got = []
    for blocks, ids in ((3, [2, 0, 1]), (nb, [nb - 1, 0, nb - 2])):
        pool = kvr.Kv4Layout(torch.empty(blocks, 1, bs // 16, kvr.KV4_TILE, dtype=torch.uint8, device=DEV),
                             _ints([ids], torch.int32))
        _append(pool, k, v, 0, 0, table)
        out = kvr.full_attn_decode_kv4(q, pos, seq, pool, table, SCALE, 3 * bs)
        at = pool.block_table[0].long()
        slots = (at[torch.arange(n, device=DEV) // bs] * bs + torch.arange(n, device=DEV) % bs)
        tiles = pool.data[at].clone()
        tiles[2, :, 3:] = 0                                                 # (positions behind the last token)
        pool.data[at] = 0
        kvr.kv4_append_rope(k, v, torch.arange(n, device=DEV), None, table, VS, pool, slots=slots)
        pages = kvr.PagedLayout(torch.empty(blocks // 2 + 2, 1, bs, 192, dtype=torch.bfloat16, device=DEV),
                                torch.empty(blocks // 2 + 2, 1, bs, 128, dtype=torch.bfloat16, device=DEV),
                                _ints([[blocks // 2 + 1, 0, 1]], torch.int32))
        kvr.kv4_unpack(pool, seq[:1], _ints([0], torch.int64), _ints([0, n], torch.int32), pages, seq[:1], T=n)
        again = pool.data[at].clone()
        r = pages.block_table[0].long()
        got.append((out, tiles[:2], again, pages.k[r].reshape(-1, 192)[:n].clone(), pages.v[r].reshape(-1, 128)[:n].clone()))
        assert torch.equal(tiles[:2], again[:2])
        del pool, pages
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert kvr.device_status() == 0
