"""The 8-bit pool on the GPU: the append's bytes against the oracle's bit for
bit, the decode against fp64 attention over the values the codes stand for, the
unpack bit for bit."""
import math

import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import kv8 as o8
from oracle.kv4 import attend

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
    """A pool with its blocks in random order and every byte `fill` (0xFF: NaN scales and full masks wherever nothing is
    written)."""
    mb = -(-max_ctx // bs)
    nb = S * mb + spare
    ids = torch.randperm(nb, generator=gen, device=DEV)[:S * mb].to(torch.int32).reshape(S, mb)
    data = torch.full((nb, hkv, bs // 16, kvr.KV8_TILE), fill, dtype=torch.uint8, device=DEV)
    return kvr.Kv8Layout(data, ids.contiguous())


def _ints(v, t):
    return torch.tensor(v, dtype=t, device=DEV)


def _append(pool, k, v, seqs, lo, rows, table, vs=VS):
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    kvr.kv8_append_rope(k, v, _ints(cu, torch.int32), _ints(lo, torch.int64), _ints(seqs, torch.int32), table, vs, pool)


def _oracle_append(data, bt, k, v, seqs, lo, rows, table, vs=VS, written=None):
    """The chunks into data by the oracle; `written`: (block, tile) -> rows there afterwards."""
    kf, vf = k.float().cpu().numpy(), v.float().cpu().numpy()
    at, bs = 0, 16 * data.shape[2]
    for s, p, n in zip(seqs, lo, rows):
        if n == 0:
            continue
        cs = table[p:p + n].cpu().numpy()
        with np.errstate(over="ignore", invalid="ignore"):
            o8.append(data, bt[s], p, o8.rope_fp32(kf[at:at + n], cs), vf[at:at + n] * np.float32(vs))
        if written is not None:
            for m in range(p // 16, (p + n - 1) // 16 + 1):
                written[int(bt[s][16 * m // bs]), 16 * m % bs // 16] = min(p + n - 16 * m, 16)
        at += n


# -- append --------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("hkv,bs", [(1, 16), (2, 64), (3, 48), (8, 128), (5, 1024)])
def test_append_bytes(table, hkv, bs):
    """Batches of chunks one after another, each sequence going on where it stood: from every place in a tile, with
    magnitudes that make scales grow or not, empty chunks between."""
    gen = _gen(100 + bs)
    rng = np.random.default_rng(bs)
    S = 5
    pool = _pool(gen, S, hkv, 2048, bs, fill=0xEE)
    want, bt = pool.data.cpu().numpy(), pool.block_table.cpu().numpy()
    held, written = [0] * S, {}
    for step in range(9):
        seqs = rng.permutation(S)[:rng.integers(1, S + 1)].tolist()
        rows = [int(r) for r in rng.choice([0, 1, 1, 2, 7, 15, 16, 17, 33, 130], len(seqs))]
        lo = [held[s] for s in seqs]
        k, v = _kv(gen, max(sum(rows), 1), hkv, 2.0)
        f = torch.exp2(torch.randint(-3, 4, (k.shape[0], 1, 1), generator=gen, device=DEV).float())
        k, v = (k.float() * f).bfloat16(), (v.float() * f.flip(0)).bfloat16()
        _append(pool, k, v, seqs, lo, rows, table)
        _oracle_append(want, bt, k, v, seqs, lo, rows, table, written=written)
        for s, r in zip(seqs, rows):
            held[s] += r
        assert kvr.device_status() == 0
        assert o8.same(pool.data.cpu().numpy(), want.copy(), written), step


def test_append_again_from_an_earlier_position(table):
    """A draft that was turned down: the sequence goes on from the draft's first position, under a scale that may have
    grown; what was behind it means nothing."""
    gen = _gen(5)
    pool = _pool(gen, 1, 2, 128, 32)
    want, bt, written = pool.data.cpu().numpy(), pool.block_table.cpu().numpy(), {}
    for lo, n, f in ((0, 20, 1.0), (20, 4, 8.0), (21, 3, 1.0), (21, 1, 0.1), (22, 30, 1.0), (32, 1, 1e-3), (16, 1, 2.0)):
        k, v = _kv(gen, n, 2)
        k, v = (k.float() * f).bfloat16(), (v.float() * f).bfloat16()
        _append(pool, k, v, [0], [lo], [n], table)
        _oracle_append(want, bt, k, v, [0], [lo], [n], table, written=written)
        for m in range((lo + n - 1) // 16 + 1, 8):
            written.setdefault((int(bt[0][16 * m // 32]), m % 2), 0)
        assert o8.same(pool.data.cpu().numpy(), want.copy(), written), (lo, n)


def test_append_corner_rows(table):
    gen = _gen(7)
    T, hkv = 48, 2
    pool = _pool(gen, 1, hkv, 64, 16, fill=0)
    k, v = _kv(gen, T, hkv)
    k[2, 1, 130] = float("nan")
    k[3, 1, 70] = float("inf")
    k[4, 0, 3] = float("-inf")                 # in a rotary pair: its partner is not finite either
    v[4, 0, 5] = float("-inf")
    v[5, 1, 64:] = float("nan")
    k[16:32, 0], v[16:32, 0] = 0.0, -0.0       # a tile of zeros
    k[16:32, 1] = (k[16:32, 1].float() * 1e-39).bfloat16()   # below fp32's normal range
    v[16:32, 1] = (v[16:32, 1].float() * 1e-36).bfloat16()
    k[32:, 0] = (k[32:, 0].float() * 1e36).bfloat16()
    k[40, 1, :64] = 3.3e38                     # finite, but not once rotated
    v[32:, 0, :] = torch.arange(128, device=DEV).bfloat16() * 0.5 / VS  # many values near half steps
    v[32:, 1] = 0.0
    v[33, 1, 9] = 1.0
    want, bt, written = pool.data.cpu().numpy(), pool.block_table.cpu().numpy(), {}
    _append(pool, k, v, [0], [0], [T], table)
    _oracle_append(want, bt, k, v, [0], [0], [T], table, written=written)
    assert o8.same(pool.data.cpu().numpy(), want, written)
    # a row that is not finite behind and ahead of others in one tile, written one by one
    pool2 = _pool(gen, 1, hkv, 64, 16, fill=0)
    for t in range(16):
        _append(pool2, k[t:t + 1].contiguous(), v[t:t + 1].contiguous(), [0], [t], [1], table)
    want2 = np.zeros_like(want)
    bt2, written2 = pool2.block_table.cpu().numpy(), {}
    for t in range(16):
        _oracle_append(want2, bt2, k[t:t + 1], v[t:t + 1], [0], [t], [1], table, written=written2)
    assert o8.same(pool2.data.cpu().numpy(), want2, written2)
    assert kvr.device_status() == 0


def test_append_scales_over_the_whole_range(table):
    """A tile per power of two from the least numbers to the greatest: quotients of 24-bit values (products with the value
    scale, rotated pairs) by 8-bit scales, rounded as the oracle's division rounds them.  Two heads and five: one head a CTA,
    and several."""
    gen = _gen(19)
    for hkv, reps in ((2, 1), (5, 6)):
        e = torch.arange(-132, 125, device=DEV).repeat(reps)
        T = 16 * len(e)
        f = torch.ldexp(torch.ones(1, device=DEV, dtype=torch.float64), e).repeat_interleave(16)[:, None, None]
        k, v = ((torch.randn(T, hkv, d, generator=gen, device=DEV).double().clamp(-3, 3) * f).bfloat16() for d in (192, 128))
        pool = _pool(gen, 1, hkv, T, 64, fill=0)
        want, bt, written = pool.data.cpu().numpy(), pool.block_table.cpu().numpy(), {}
        _append(pool, k, v, [0], [0], [T], table)
        _oracle_append(want, bt, k, v, [0], [0], [T], table, written=written)
        assert o8.same(pool.data.cpu().numpy(), want, written)
    assert kvr.device_status() == 0


def test_append_halves_round_to_even(table):
    """Keys that lie exactly between two codes: bf16 values over a bf16 scale."""
    T = 16
    k = torch.zeros(T, 1, 192, device=DEV)
    k[:, 0, 64:] = (torch.arange(128, device=DEV).float() - 63.5) * 1.0       # scale 1 where the largest is 127
    k[0, 0, 64] = 127.0
    v = torch.zeros(T, 1, 128, device=DEV)
    v[:, 0] = (torch.arange(128, device=DEV).float() - 64) * 1.5
    v[0, 0, 0] = 381.0                                                        # scale 3: every odd multiple of 1.5 is a half
    k, v = k.bfloat16(), v.bfloat16()
    pool = _pool(_gen(1), 1, 1, 16, 16, fill=0)
    want, written = pool.data.cpu().numpy(), {}
    _append(pool, k, v, [0], [0], [T], table, vs=1.0)
    _oracle_append(want, pool.block_table.cpu().numpy(), k, v, [0], [0], [T], table, vs=1.0, written=written)
    assert o8.scales(want[int(pool.block_table[0, 0]), 0, 0]).tolist() == [1.0, 3.0]
    assert np.array_equal(pool.data.cpu().numpy(), want)


@pytest.mark.parametrize("n", [1, 63, 65, 100, 2049, 5000])
def test_append_many_chunks(table, n):
    """Chunks are found by a search over cu_rows, in rounds for more than 64 of them."""
    gen = _gen(n)
    rng = np.random.default_rng(n)
    rows = rng.choice([0, 1, 1, 1, 2, 5, 40], n).tolist()
    lo = rng.integers(0, 20, n).tolist()
    lo = [16 * (x // 16) for x in lo]
    pool = _pool(gen, n, 1, 64, 16, fill=0)
    T = max(sum(rows), 1)
    k, v = _kv(gen, T, 1)
    _append(pool, k, v, list(range(n)), lo, rows, table)
    out = kvr.LinearLayout.empty(T, 1)
    cu = _ints(np.concatenate([[0], np.cumsum(rows)]).tolist(), torch.int32)
    kvr.kv8_unpack(pool, torch.arange(n, dtype=torch.int32, device=DEV), _ints(lo, torch.int64), cu, out)
    assert kvr.device_status() == 0
    # what comes back is within half a step of what went in, the step at most (1 + 2^-7) of max |x| / 127, and bf16's half step
    c = cu.tolist()
    kk, vv = k.float().cpu().numpy(), v.float().cpu().numpy()
    gk, gv = out.k.float().cpu().numpy(), out.v.float().cpu().numpy()
    for i in range(n):
        if rows[i]:
            a, b = c[i], c[i + 1]
            x = o8.rope_fp32(kk[a:b], table[lo[i]:lo[i] + rows[i]].cpu().numpy())
            for got, ref in ((gk[a:b], x), (gv[a:b], vv[a:b] * np.float32(VS))):
                m = np.abs(ref).max()
                assert np.abs(got - ref).max() <= m * (1 + 2.0 ** -7) / 254 + 2.0 ** -8 * m, i


@pytest.mark.parametrize("n,long", [(1, 1), (70, 60), (70, 0), (1500, 40), (1500, 0)])
def test_append_short_chunks(table, n, long):
    """Chunks of none to three rows behind what each sequence holds, over the ends of tiles, with padding between, and (as
    long as the mean stays near one) a long one among them: the oracle's bytes."""
    gen, rng = _gen(n + long), np.random.default_rng(n + long)
    hkv = 2
    first = rng.integers(0, 20, n)
    rows = rng.choice([0, 1, 1, 1, 2, 3], n)
    rows[n // 2] = max(long, 1)
    cap = int((first + rows).max()) + 1
    pool = _pool(gen, n, hkv, cap, 16, fill=0)
    want, bt, written = pool.data.cpu().numpy(), pool.block_table.cpu().numpy(), {}
    ids = rng.permutation(n)
    gone = [i for i in range(n) if n > 1 and rng.random() < 0.1]
    for lo, cnt in ((np.zeros(n, int), first), (first, rows)):
        T = max(int(cnt.sum()), 1)
        k, v = _kv(gen, T, hkv)
        seqs = np.where(np.isin(np.arange(n), gone) & (cnt is rows), -1, ids)
        _append(pool, k, v, seqs.tolist(), lo.tolist(), cnt.tolist(), table)
        at = np.concatenate([[0], np.cumsum(cnt)])
        for i in range(n):
            if seqs[i] >= 0:
                _oracle_append(want, bt, k[at[i]:at[i + 1]], v[at[i]:at[i + 1]], [int(seqs[i])], [int(lo[i])], [int(cnt[i])],
                               table, written=written)
    assert T <= T // 16 + 2 * n
    assert kvr.device_status() == 0
    assert o8.same(pool.data.cpu().numpy(), want, written)


def test_append_padding_and_flags(table):
    gen = _gen(11)
    hkv, bs = 2, 32
    pool = _pool(gen, 4, hkv, 64, bs, fill=0x11)
    pool.block_table[3, 1] = pool.num_blocks
    before = pool.data.clone()
    k, v = _kv(gen, 12, hkv)

    def run(seqs, lo, cu):
        kvr.kv8_append_rope(k, v, _ints(cu, torch.int32), _ints(lo, torch.int64), _ints(seqs, torch.int32), table, VS, pool)
        return kvr.device_status()

    assert run([-1, -1], [0, 1 << 60], [0, 4, 12]) == 0                              # padding, whatever its position
    assert run([4, -2], [0, 0], [0, 4, 8]) == kvr.DEV_BAD_SEQ
    assert run([0, 1, 2], [-1, 61, 1 << 40], [0, 4, 8, 12]) == kvr.DEV_BAD_POS        # 64 positions a sequence
    assert run([0], [-(1 << 62)], [0, 4]) == kvr.DEV_BAD_POS
    assert run([3], [32], [0, 4]) == kvr.DEV_BAD_BLOCK
    assert run([0], [0], [5, 3]) == kvr.DEV_BAD_ROWS and run([0], [0], [0, 13]) == kvr.DEV_BAD_ROWS
    assert run([0], [0], [-3, 3]) == kvr.DEV_BAD_ROWS
    assert torch.equal(pool.data, before)
    # good chunks beside bad ones are written, rows behind the last chunk are not looked at
    assert run([7, 1, -1, 0], [0, 3, 0, 16], [0, 2, 5, 6, 8]) == kvr.DEV_BAD_SEQ
    want, written = before.cpu().numpy(), {}
    bt = pool.block_table.cpu().numpy()
    _oracle_append(want, bt, k[2:5], v[2:5], [1], [3], [3], table, written=written)
    _oracle_append(want, bt, k[6:8], v[6:8], [0], [16], [2], table, written=written)
    assert o8.same(pool.data.cpu().numpy(), want, written)


# -- decode --------------------------------------------------------------------------------------------------------------

def _check_decode(got, q, pos, seq, pool, table, what="", rel_bar=True, least=0.0):
    """Every row against fp64.  The output is rounded by half a bf16 step, 2^-8 |o| at most.  A score moves by at most
    2^-11 sum |q||k| for the rounding of the rotated q to fp16, and by less than as much again for what is held in fp32
    (12 products whose sums are cut off at 2^-23, the scale's factor): 2^-10 sum |q||k|, of which a weight and the sum
    of weights each move by the exponential.  A weight is rounded to fp16 once, 2^-11 of it, and what is below fp16's
    least normal number by 2^-36 of the largest share, n keys of them; the sums over keys are cut off below 2^-23, once
    a tile: together under 2^-10 of sum p |v| and 2^-20 |v|_max (n < 2^16, a thousand tiles a warp)."""
    data, bt = pool.data.cpu().numpy(), pool.block_table.cpu().numpy()
    G = q.shape[1] // pool.num_kv_heads
    qf, g = q.float().cpu().numpy(), got.double().cpu().numpy()
    cache = {}
    for b, (p, s) in enumerate(zip(pos, seq)):
        for h in range(pool.num_kv_heads):
            if (s, h) not in cache:
                n = max(pp for pp, ss in zip(pos, seq) if ss == s) + 1
                cache[s, h] = o8.sequence(data, bt[s], h, n)
            K, V, ok = cache[s, h]
            hs = slice(h * G, (h + 1) * G)
            want, a, w = attend(qf[b, hs], p, K, V, ok, table[p].cpu().numpy(), SCALE)
            err = np.abs(g[b, hs] - want)
            vmax = np.abs(V[:p + 1][ok[:p + 1]]).max() if ok[:p + 1].any() else 0.0
            move = np.exp(2 * 2.0 ** -10 * a[:, None]) - 1
            tol = 2.0 ** -8 * np.abs(want) + move * (w + np.abs(want)) + 2.0 ** -10 * w + 2.0 ** -20 * vmax + least
            assert np.all(err <= tol), f"{what} row {b} head {h}: {np.max(err - tol):.3e} over"
            if rel_bar:
                rel = np.sqrt((err ** 2).mean(1) / np.maximum((want ** 2).mean(1), 1e-300))
                assert rel.max() <= 1e-2, f"{what} row {b} head {h}: rel RMS {rel.max():.3e}"


def _filled(gen, lens, hkv, bs, table, shift=0.0, max_ctx=None):
    pool = _pool(gen, len(lens), hkv, max_ctx or max(lens), bs)
    k, v = _kv(gen, sum(lens), hkv, shift)
    _append(pool, k, v, list(range(len(lens))), [0] * len(lens), lens, table)
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
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, 1000)
    assert kvr.device_status() == 0
    _check_decode(out, q, pos, seq, pool, table)


@pytest.mark.parametrize("G", [2, 8, 12, 16])
@pytest.mark.parametrize("B,hkv,max_ctx", [(1, 1, 1), (1, 2, 513), (3, 1, 1024), (40, 2, 1025), (2, 4, 2048), (70, 2, 1030),
                                           (5, 1, 2049), (300, 1, 200)])
def test_decode_forms(table, B, hkv, max_ctx, G):
    """Either side of the sizes at which a call goes by clusters in one launch, and batches that are planned by a kernel
    of their own."""
    gen = _gen(B + max_ctx + G)
    lens = torch.randint(1, max_ctx + 1, (B,), generator=gen, device=DEV).tolist()
    lens[0] = max_ctx
    pool = _filled(gen, lens, hkv, 64, table, max_ctx=max_ctx)
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pos, seq = [n - 1 for n in lens], list(range(B))
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, max_ctx)
    assert kvr.device_status() == 0
    few = list(range(min(B, 6)))
    _check_decode(out[few], q[few], pos[:6], seq[:6], pool, table)
    # the same rows among longer ones (the other form): the same numbers but for the order of the sums
    if B <= 5:
        wide = torch.full((B, -(-9000 // 64)), -1, dtype=torch.int32, device=DEV)
        wide[:, :pool.max_blocks] = pool.block_table
        pool2 = kvr.Kv8Layout(pool.data, wide)
        out2 = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool2, table, SCALE, 9000)
        _check_decode(out2[few], q[few], pos[:6], seq[:6], pool2, table)


@pytest.mark.parametrize("ctx,hkv,G,dist", [(8193, 1, 16, 0.0), (20001, 2, 16, 3.0), (65535, 1, 8, 1.0)])
def test_decode_long(table, ctx, hkv, G, dist):
    gen = _gen(ctx)
    pool = _filled(gen, [ctx], hkv, 64, table, shift=dist)
    q = (torch.randn(2, hkv * G, 192, generator=gen, device=DEV) * 2).bfloat16()
    pos = [ctx - 1, ctx // 2]
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints([0, 0], torch.int32), pool, table, SCALE, ctx)
    _check_decode(out, q, pos, [0, 0], pool, table)
    assert kvr.device_status() == 0


def test_decode_draft_rows_share_a_sequence(table):
    gen = _gen(31)
    lens, C, hkv, G = [70, 300, 1025], 4, 2, 8
    pool = _filled(gen, lens, hkv, 32, table)
    pos = [n - C + c for n in lens for c in range(C)]
    seq = [s for s in range(len(lens)) for _ in range(C)]
    q = torch.randn(len(pos), hkv * G, 192, generator=gen, device=DEV).bfloat16()
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, 1025)
    _check_decode(out, q, pos, seq, pool, table)


@pytest.mark.parametrize("most", [1025, 9000])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 8, 9, 16])
def test_decode_rows_of_one_sequence_go_together(table, G, most):
    """Neighbouring rows of one sequence are taken together, in aligned blocks of the batch: drafts of every length at
    every place of a block, rows far apart or in any order, the same row twice, rows that cannot be served between, a
    sequence that comes again later."""
    gen = _gen(33 + G)
    lens, hkv = [70, 300, 1025, 5, 16], 2
    pool = _filled(gen, lens, hkv, 32, table, max_ctx=most)
    rows = [(0, 66), (0, 67), (0, 68), (1, 299), (2, 1020), (2, 1021), (2, 1022), (2, 1023), (2, 1024), (2, 0), (2, 1024),
            (2, 1024), (9, 5), (2, 512), (2, most), (2, 3), (3, 0), (3, 4), (4, 15), (-1, 0), (4, 14), (4, 14), (1, 16), (1, 15),
            (1, 31), (0, 69), (0, 0), (2, 15), (2, 16), (2, 700), (2, 17)]
    q = torch.randn(len(rows), hkv * G, 192, generator=gen, device=DEV).bfloat16()
    out = torch.full((len(rows), hkv * G, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    kvr.full_attn_decode_kv8(q, _ints([p for _, p in rows], torch.int64), _ints([s for s, _ in rows], torch.int32), pool, table,
                             SCALE, most, out=out)
    assert kvr.device_status() == kvr.DEV_BAD_POS | kvr.DEV_BAD_SEQ
    bad = [i for i, (s, p) in enumerate(rows) if not 0 <= s < 5 or p >= most]
    assert len(bad) == 3 and not out[bad].any()
    good = [i for i in range(len(rows)) if i not in bad]
    _check_decode(out[good], q[good], [rows[i][1] for i in good], [rows[i][0] for i in good], pool, table)
    # a NaN in a key or value row reaches exactly the rows that see it, a NaN in a query its own head
    k, v = _kv(gen, 1025 - 700, hkv)
    k[0, 0, 100] = v[1, 1, 3] = float("nan")      # positions 700 and 701 of sequence 2
    _append(pool, k, v, [2], [700], [325], table)
    q[5, hkv * G - 1, 64] = float("inf")
    out = kvr.full_attn_decode_kv8(q, _ints([p for _, p in rows], torch.int64), _ints([s for s, _ in rows], torch.int32), pool,
                                   table, SCALE, most)
    kvr.device_status()
    want = torch.zeros_like(out, dtype=torch.bool)
    for i, (s, p) in enumerate(rows):
        if s == 2 and i not in bad:
            want[i, :G] = p >= 700
            want[i, G:] = p >= 701
    want[5, -1] = True
    assert torch.equal(torch.isnan(out), want)


@pytest.mark.parametrize("G,hkv,most", [(8, 2, 2300), (16, 1, 2300), (4, 1, 700)])
def test_decode_thousands_of_rows(table, G, hkv, most):
    """2600 rows, by a plan of their own: one to four neighbours of a sequence, and rows that cannot be served between."""
    gen, rng = _gen(53), np.random.default_rng(53)
    S, B = 40, 2600
    lens = rng.integers(5, most, S).tolist()
    pool = _filled(gen, lens, hkv, 32, table, max_ctx=most)
    seq, pos = [], []
    while len(seq) < B:
        s = int(rng.integers(0, S))
        for _ in range(int(rng.integers(1, 5))):
            seq.append(s)
            pos.append(int(rng.integers(0, lens[s])))
        if rng.random() < 0.05:
            seq[-1] = S if rng.random() < 0.5 else -1
        elif rng.random() < 0.05:
            pos[-1] = -1
    seq, pos = seq[:B], pos[:B]
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, most)
    assert kvr.device_status() == (kvr.DEV_BAD_SEQ | kvr.DEV_BAD_POS)
    bad = [b for b in range(B) if not 0 <= seq[b] < S or pos[b] < 0]
    assert len(bad) > 20 and not out[bad].any()
    few = [b for b in range(B) if b not in set(bad)][::9]
    _check_decode(out[few], q[few], [pos[b] for b in few], [seq[b] for b in few], pool, table)
    again = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, most)
    kvr.device_status()
    assert torch.equal(out, again)


@pytest.mark.parametrize("C,G,B", [(2, 16, 9), (3, 8, 70), (4, 4, 40), (4, 16, 70)])
def test_decode_drafts_of_long_contexts(table, C, G, B):
    """Drafts of many sequences, on the work line, planned by the split kernel's CTAs or by a kernel of their own."""
    gen = _gen(C * G + B)
    hkv = 2
    lens = torch.randint(C, 6000, (B,), generator=gen, device=DEV).tolist()
    pool = _filled(gen, lens, hkv, 64, table, max_ctx=6000)
    pos = [n - C + c for n in lens for c in range(C)]
    seq = [s for s in range(B) for _ in range(C)]
    q = torch.randn(B * C, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, 6000)
    assert kvr.device_status() == 0
    few = list(range(3 * C)) + list(range(B * C - 2 * C, B * C))
    _check_decode(out[few], q[few], [pos[i] for i in few], [seq[i] for i in few], pool, table)


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("vscales", [(1e-6,), (2e4,), (1.0, 1e-5, 3e3, 1e-2), (1e-3, 6e4), (1e-30, 1.0, 1e28), (0.0, 1.0)])
def test_decode_value_scales_apart(table, vscales, G):
    """Values whose scales differ by orders of magnitude from tile to tile, in both orders of appearance."""
    gen = _gen(41)
    n, hkv = 600, 1
    for flip in (False, True):
        pool = _pool(gen, 1, hkv, n, 64)
        k, v = _kv(gen, n, hkv)
        f = torch.tensor(vscales, device=DEV).repeat_interleave(48).repeat(14)[:n]
        f = f.flip(0) if flip else f
        _append(pool, k, (v.float() * f[:, None, None]).bfloat16(), [0], [0], [n], table)
        q = torch.randn(1, hkv * G, 192, generator=gen, device=DEV).bfloat16()
        out = kvr.full_attn_decode_kv8(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
        _check_decode(out, q, [n - 1], [0], pool, table, f"{vscales} {flip}")


@pytest.mark.parametrize("G,rows", [(8, 1), (16, 1), (8, 4)])
@pytest.mark.parametrize("n", [600, 9000])
@pytest.mark.parametrize("mag", [1e-32, 1e-34, 1e-36, 1e-37])
def test_decode_values_near_the_least_numbers(table, mag, n, G, rows):
    """Scales down to the numbers below 2^-126.  Beside _check_decode's terms, an output below 2^-126 is rounded by half
    of bf16's least step there, 2^-134."""
    gen = _gen(43)
    pool = _pool(gen, 1, 1, n, 64)
    k, v = _kv(gen, n, 1)
    _append(pool, k, (v.float() * mag).bfloat16(), [0], [0], [n], table)
    q = torch.randn(rows, G, 192, generator=gen, device=DEV).bfloat16() * 3
    pos = [n - rows + i for i in range(rows)]
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints([0] * rows, torch.int32), pool, table, SCALE, n)
    _check_decode(out, q, pos, [0] * rows, pool, table, f"{mag}", rel_bar=False, least=2.0 ** -134)
    assert torch.count_nonzero(out) > 0.9 * out.numel()


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("small,large", [(1e-6, 1e3), (1e-12, 1.0), (1.0, 1e20)])
def test_decode_light_keys_of_large_values_and_heavy_ones_of_small(table, G, small, large):
    """Each half of the keys has half of the output: the heavy ones have small values, the light ones large, in either
    order.  A weight that were rounded beside the largest probability alone, or beside the largest value, would be lost."""
    gen = _gen(43)
    n = 512
    gap = math.log(large / small) / SCALE  # of the scores before scaling
    for flip in (False, True):
        pool = _pool(gen, 1, 1, n, 64)
        u = torch.zeros(192, device=DEV)
        u[64 + 17] = 1.0
        heavy = (torch.arange(n, device=DEV) // 16 % 2 == 0) != flip
        k = (torch.randn(n, 192, generator=gen, device=DEV) * 0.02 + torch.where(heavy, gap / 16, 0.0)[:, None] * u).bfloat16()
        v = torch.rand(n, 128, generator=gen, device=DEV) + 0.5
        v = (v * torch.where(heavy, small, large)[:, None]).bfloat16()
        _append(pool, k[:, None].contiguous(), v[:, None].contiguous(), [0], [0], [n], table)
        q = (torch.randn(1, G, 192, generator=gen, device=DEV) * 0.02 + 16 * u).bfloat16()
        out = kvr.full_attn_decode_kv8(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
        _check_decode(out, q, [n - 1], [0], pool, table, f"flip {flip}", rel_bar=False)
        # and both halves are there: without the heavy ones (or the light) the output would be off by far more than the bound
        K, V, ok = o8.sequence(pool.data.cpu().numpy(), pool.block_table[0].cpu().numpy(), 0, n)
        hv = heavy.cpu().numpy()
        both, a, w = attend(q[0].float().cpu().numpy(), n - 1, K, V, ok, table[n - 1].cpu().numpy(), SCALE)
        part, _, _ = attend(q[0].float().cpu().numpy(), n - 1, K, np.where(hv[:, None], V, 0), ok, table[n - 1].cpu().numpy(), SCALE)
        share = part / both
        assert 0.02 < share.min() and share.max() < 0.98


@pytest.mark.parametrize("mag", [0.0, 1e-30, 1e-3, 30.0, 1e4])
def test_decode_query_magnitudes(table, mag):
    """Queries of any size: zeros (all keys weigh the same), tiny, and so large that one key takes everything."""
    gen = _gen(43)
    n, hkv, G = 200, 2, 4
    pool = _filled(gen, [n], hkv, 64, table)
    q = (torch.randn(1, hkv * G, 192, generator=gen, device=DEV) * mag).bfloat16()
    out = kvr.full_attn_decode_kv8(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
    if mag < 1e3:
        _check_decode(out, q, [n - 1], [0], pool, table, rel_bar=mag < 10)
    else:  # the weights are one key's or split by rounding between near ties: between the least and largest values
        assert torch.isfinite(out).all()
        for h in range(hkv):
            _, V, _ = o8.sequence(pool.data.cpu().numpy(), pool.block_table[0].cpu().numpy(), h, n)
            o = out[0, h * G:(h + 1) * G].double().cpu().numpy()
            room = 2.0 ** -7 * np.abs(V).max(0)
            assert (o <= V.max(0) + room).all() and (o >= V.min(0) - room).all()


@pytest.mark.parametrize("G", [8, 16])
def test_decode_scores_rise_and_fall(table, G):
    """Scores that climb along the keys (every tile raises the maximum) and that fall by hundreds (late keys weigh
    nothing), and one far above the rest at either end."""
    gen = _gen(47)
    n = 1500
    u = torch.zeros(192, device=DEV)
    u[64:] = torch.randn(128, generator=gen, device=DEV)
    u /= u.norm()
    for ramp in (torch.linspace(-300, 300, n), torch.linspace(300, -300, n), torch.eye(n)[0] * 400, torch.eye(n)[-1] * 400):
        pool = _pool(gen, 1, 1, n, 64)
        k, v = _kv(gen, n, 1)
        k = (k.float() * 0.05 + ramp.to(DEV)[:, None, None] * u * 0.5).bfloat16()
        _append(pool, k, v, [0], [0], [n], table)
        q = (torch.randn(1, G, 192, generator=gen, device=DEV) * 0.1 + u * 14).bfloat16()
        out = kvr.full_attn_decode_kv8(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
        # scores of hundreds carry the fp16 rounding of q, so the bound is wide here and the rel RMS bar does not apply
        _check_decode(out, q, [n - 1], [0], pool, table, rel_bar=False)


@pytest.mark.parametrize("G", [4, 12])
def test_decode_nan_and_what_lies_behind(table, G):
    gen = _gen(53)
    n, hkv = 100, 2
    pool = _filled(gen, [n, n], hkv, 16, table)   # 0xFF (NaN scales, full masks) wherever nothing was written
    k, v = _kv(gen, 1, hkv)
    v[0, 1, 70] = float("nan")                    # the last key of sequence 0, KV head 1
    _append(pool, k, v, [0], [n - 1], [1], table)
    k2, v2 = _kv(gen, 60, hkv)
    k2[0, 0, 0] = float("inf")                    # a key of KV head 0 of sequence 1, and what follows it written again
    _append(pool, k2, v2, [1], [40], [60], table)
    q = torch.randn(2, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pos, seq = _ints([n - 1, n - 1], torch.int64), _ints([0, 1], torch.int32)
    for most in (n, None):
        lay = pool
        if most is None:                          # the other form
            wide = torch.full((2, 600), -1, dtype=torch.int32, device=DEV)
            wide[:, :pool.max_blocks] = pool.block_table
            lay, most = kvr.Kv8Layout(pool.data, wide), 9600
        out = kvr.full_attn_decode_kv8(q, pos, seq, lay, table, SCALE, most)
        nan = torch.isnan(out)
        want = torch.zeros_like(nan)
        want[0, G:] = True
        want[1, :G] = True
        assert torch.equal(nan, want)
        # queries before the bad rows do not see them, though they share a tile with them
        out = kvr.full_attn_decode_kv8(q, _ints([n - 2, 39], torch.int64), seq, lay, table, SCALE, most)
        _check_decode(out, q, [n - 2, 39], [0, 1], lay, table)
        # a query holding a NaN or an infinity spoils its own head only
        q3 = q.clone()
        q3[0, 1, 3] = float("nan")
        q3[0, 2, 100] = float("inf")
        out = kvr.full_attn_decode_kv8(q3, _ints([n - 2, 39], torch.int64), seq, lay, table, SCALE, most)
        bad = torch.zeros_like(nan)
        bad[0, 1:3] = True
        assert torch.equal(torch.isnan(out), bad)
    assert kvr.device_status() == 0


@pytest.mark.parametrize("most", [200, 9000])
def test_decode_bad_rows_and_blocks(table, most):
    gen = _gen(59)
    n, hkv, G = 200, 2, 8
    pool = _filled(gen, [n] * 5, hkv, 32, table, max_ctx=most)
    pool.block_table[1, 2] = -1
    pool.block_table[2, 0] = pool.num_blocks
    pool.block_table[4, :] = -7
    q = torch.randn(7, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    seq = [0, 1, 2, 9, -1, 3, 4]
    pos = [n - 1, n - 1, n - 1, 5, 5, most, n - 1]
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, most,
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
    first = kvr.full_attn_decode_kv8(q, pos, seq, pool, table, SCALE, 4096)
    for _ in range(5):
        assert torch.equal(kvr.full_attn_decode_kv8(q, pos, seq, pool, table, SCALE, 4096), first)
    # two captured graphs on two streams, each with a workspace of its own, replayed side by side with other lengths
    n = kvr.full_attn_decode_kv8_workspace_size(3, hkv * G, hkv, 4096)
    runs = []
    for i in range(2):
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        p, out = pos.clone(), torch.empty_like(first)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            kvr.full_attn_decode_kv8(q, p, seq, pool, table, SCALE, 4096, workspace=ws, out=out)
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
    pool = kvr.Kv8Layout(pool.data, pool.block_table[torch.arange(B, device=DEV) % 3].contiguous())
    q = torch.randn(B, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    own = torch.zeros(B, ctx // bs, dtype=torch.int32, device=DEV)
    free, left = torch.zeros(B, dtype=torch.int32, device=DEV), _ints([B], torch.int32)
    cu, count = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    pos, slots = torch.zeros(B, dtype=torch.int64, device=DEV), torch.empty(B, dtype=torch.int64, device=DEV)
    seq, add = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    ws = torch.empty(kvr.full_attn_decode_kv8_workspace_size(B, hkv * G, hkv, ctx), dtype=torch.uint8, device=DEV)
    steps = []
    for _ in range(12):
        lens = torch.randint(0, 200, (B,), generator=gen, device=DEV)
        lens[torch.randint(0, B, (2,), generator=gen, device=DEV)] = torch.randint(0, ctx, (2,), generator=gen, device=DEV)
        steps.append((lens, torch.randperm(B, generator=gen, device=DEV).to(torch.int32),
                      torch.empty(B, hkv * G, 128, dtype=torch.bfloat16, device=DEV)))
    torch.cuda.synchronize()
    for lens, ids, out in steps:
        kvr.kv_pages_grow(own, 1, bs, ids, lens, add, free, left, cu, pos, seq, slots, free_count_out=count)
        kvr.full_attn_decode_kv8(q, pos, seq, pool, table, SCALE, ctx, workspace=ws, out=out)
    torch.cuda.synchronize()
    for lens, ids, out in steps:
        assert torch.equal(out, kvr.full_attn_decode_kv8(q, lens, ids, pool, table, SCALE, ctx))
    assert kvr.device_status() == 0
    lens, ids, out = steps[-1]
    few = [0, 1, 2]
    _check_decode(out[few], q[few], lens[few].tolist(), ids[few].tolist(), pool, table)


@pytest.mark.parametrize("ctx,G", [(513, 4), (9000, 4), (9000, 16)])
def test_decode_stalled_wait_leaves_in_time(table, ctx, G):
    gen = _gen(67)
    pool = _filled(gen, [ctx], 2, 64, table)
    q = torch.randn(1, 2 * G, 192, generator=gen, device=DEV).bfloat16()
    args = (q, _ints([ctx - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, ctx)
    first = kvr.full_attn_decode_kv8(*args)
    torch.cuda.synchronize()
    kvr.debug_stall_next(1, 2_000_000)
    kvr.full_attn_decode_kv8(*args)
    assert kvr.device_status() == kvr.DEV_TIMEOUT
    assert torch.equal(kvr.full_attn_decode_kv8(*args), first)
    assert kvr.device_status() == 0


def test_calls_on_another_stream(table):
    gen = _gen(71)
    n, hkv, G = 5000, 2, 8
    k, v = _kv(gen, n, hkv)
    q = torch.randn(1, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    pool = _pool(gen, 1, hkv, n, 64)
    rows = kvr.LinearLayout.empty(n, hkv)
    cu, zero, seq = _ints([0, n], torch.int32), _ints([0], torch.int64), _ints([0], torch.int32)
    pos = _ints([n - 1], torch.int64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kvr.kv8_append_rope(k, v, cu, zero, seq, table, VS, pool, stream=st)
    out = kvr.full_attn_decode_kv8(q, pos, seq, pool, table, SCALE, n, stream=st)
    kvr.kv8_unpack(pool, seq, zero, cu, rows, stream=st)
    st.synchronize()
    _check_decode(out, q, [n - 1], [0], pool, table)
    wk, wv = _want_unpacked(pool, 0, 0, n)
    assert torch.equal(rows.k.cpu(), wk) and torch.equal(rows.v.cpu(), wv)


def test_two_streams_at_once(table):
    """Two streams, each with a pool, rows and a workspace of its own, go on at the same time: as one after the other."""
    hkv, G, n, steps = 2, 8, 2500, 12

    def prepare(seed):
        gen = _gen(seed)
        lens = [n, 700, 1300]
        pool = _filled(gen, lens, hkv, 64, table, max_ctx=n + 3 * steps)
        kv = [_kv(gen, 6, hkv) for _ in range(steps)]
        q = [torch.randn(6, hkv * G, 192, generator=gen, device=DEV).bfloat16() for _ in range(steps)]
        most = pool.max_blocks * 64
        ws = torch.empty(kvr.full_attn_decode_kv8_workspace_size(6, hkv * G, hkv, most), dtype=torch.uint8, device=DEV)
        rows = kvr.LinearLayout.empty(sum(lens) + 3 * 3 * steps, hkv)
        out = [torch.empty(6, hkv * G, 128, dtype=torch.bfloat16, device=DEV) for _ in range(steps)]
        batch = []
        for i in range(steps):
            at = [x + 2 * i for x in lens]
            batch.append((_ints([0, 2, 4, 6], torch.int32), _ints(at, torch.int64), _ints([a + j for a in at for j in (0, 1)], torch.int64)))
        ids, each = _ints([0, 1, 2], torch.int32), _ints([0, 0, 1, 1, 2, 2], torch.int32)
        end = _ints(np.concatenate([[0], np.cumsum([x + 2 * steps for x in lens])]).tolist(), torch.int32)
        return pool, kv, q, ws, rows, out, batch, ids, each, end, _ints([0, 0, 0], torch.int64), most

    def step(x, i, st):
        pool, kv, q, ws, rows, out, batch, ids, each, end, zero, most = x
        cu, at, pos = batch[i]
        kvr.kv8_append_rope(*kv[i], cu, at, ids, table, VS, pool, stream=st)
        kvr.full_attn_decode_kv8(q[i], pos, each, pool, table, SCALE, most, workspace=ws, out=out[i], stream=st)
        if i + 1 == steps:
            kvr.kv8_unpack(pool, ids, zero, end, rows, stream=st)

    def results(x):
        n = int(x[9][-1])
        return [*x[5], x[4].k[:n], x[4].v[:n]]

    alone = []
    for seed in (81, 82):
        x = prepare(seed)
        for i in range(steps):
            step(x, i, None)
        torch.cuda.synchronize()
        alone.append(results(x))
    both, streams = [prepare(81), prepare(82)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(steps):
        for x, st in zip(both, streams):
            step(x, i, st)
    torch.cuda.synchronize()
    assert kvr.device_status() == 0
    for x, want in zip(both, alone):
        for a, b in zip(results(x), want):
            assert torch.equal(a, b)


def test_arrays_that_start_16_bytes_off(table):
    """Every array at the least alignment that the calls ask for: the same bytes as on aligned ones."""
    gen = _gen(83)
    n, hkv, G = 900, 3, 8
    k, v = _kv(gen, n, hkv)
    q = torch.randn(2, hkv * G, 192, generator=gen, device=DEV).bfloat16()

    def off(t):
        words = 16 // t.element_size()
        return torch.cat([t.new_zeros(words), t.reshape(-1)])[words:].view(t.shape)

    def run(put):
        pool = _pool(_gen(84), 1, hkv, n, 48, fill=0)
        pool = kvr.Kv8Layout(put(pool.data), pool.block_table)
        cs = put(table[:n].contiguous())
        cu, zero, seq = _ints([0, 7, n], torch.int32), _ints([0, 7], torch.int64), _ints([0, 0], torch.int32)
        kvr.kv8_append_rope(put(k[:7]), put(v[:7]), cu[:2].contiguous(), zero[:1].contiguous(), seq[:1].contiguous(), cs, VS, pool)
        kvr.kv8_append_rope(put(k[7:]), put(v[7:]), _ints([0, n - 7], torch.int32), zero[1:].contiguous(), seq[:1].contiguous(),
                            cs, VS, pool)
        res = [pool.data]
        res.append(kvr.full_attn_decode_kv8(put(q), _ints([n - 1, 400], torch.int64), seq, pool, cs, SCALE, n,
                                            out=put(q.new_zeros(2, hkv * G, 128))))
        rows = kvr.LinearLayout(put(k.new_zeros(n, hkv, 192)), put(k.new_zeros(n, hkv, 128)))
        kvr.kv8_unpack(pool, seq[:1].contiguous(), zero[:1].contiguous(), _ints([0, n], torch.int32), rows)
        return res + [rows.k, rows.v]

    for a, b in zip(run(off), run(lambda t: t.clone())):
        assert torch.equal(a, b)
    assert kvr.device_status() == 0


# -- long ----------------------------------------------------------------------------------------------------------------

def _values_gpu(tiles):
    """Tiles [n, 5136] -> K [16 n, 192], V [16 n, 128] in fp64, on the GPU."""
    K = torch.empty(tiles.shape[0], 16, 192, dtype=torch.float64, device=DEV)
    V = torch.empty(tiles.shape[0], 16, 128, dtype=torch.float64, device=DEV)
    s = tiles[:, 5120:5128].contiguous().view(torch.float32).double()
    for r in range(16):
        kc, vc = o8.places(r)
        K[:, r] = (tiles[:, torch.from_numpy(kc).to(DEV)].double() - 128) * s[:, :1]
        V[:, r] = (tiles[:, torch.from_numpy(vc).to(DEV)].double() - 128) * s[:, 1:]
    return K.flatten(0, 1), V.flatten(0, 1)


def _tiles(gen, n, ks, vs):
    """n tiles of random codes in -127..127 under given scales [n] or numbers."""
    t = torch.randint(1, 256, (n, kvr.KV8_TILE), generator=gen, device=DEV, dtype=torch.uint8)
    tail = torch.zeros(n, 4, device=DEV)
    tail[:, 0], tail[:, 1] = ks, vs
    t[:, 5120:] = tail.view(torch.uint8)
    return t


@pytest.mark.parametrize("G", [8, 16])
def test_decode_a_million_keys(G):
    """One row of 2^20 keys and a few, every weight alike: the sums stay exact to their rounding over the longest pieces."""
    gen = _gen(81)
    n = (1 << 20) + 37
    nt = -(-n // 16)
    data = _tiles(gen, -(-nt // 4) * 4, 2.0 ** -9, 2.0 ** -5).view(-1, 1, 4, kvr.KV8_TILE)
    table = torch.zeros(n, 32, 2, device=DEV)
    table[..., 0] = 1.0
    pool = kvr.Kv8Layout(data, torch.arange(data.shape[0], dtype=torch.int32, device=DEV)[None])
    q = torch.randn(1, G, 192, generator=gen, device=DEV).bfloat16()
    out = kvr.full_attn_decode_kv8(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
    K, V = _values_gpu(data.view(-1, kvr.KV8_TILE))
    K, V = K[:n], V[:n]
    x = q[0].double()
    w = torch.softmax(x @ K.T * SCALE, -1)
    want, wv = w @ V, w @ V.abs()
    err = (out[0].double() - want).abs()
    # a score moves by 2^-11 of what it adds up, of either sign and at random over 10^6 keys; 2^-11 of a weight, likewise:
    # three deviations of both, and the worst of it for the sums cut off at 2^-23 every tile (up to 2048 a warp)
    a = (x.abs() @ K.abs().T * SCALE).amax(1, keepdim=True)
    rms = (w * w) @ (V * V)
    tol = 2.0 ** -8 * want.abs() + 6 * (2.0 ** -10 * a + 2.0 ** -10) * rms.sqrt() + 2.0 ** -12 * wv
    assert torch.all(err <= tol), float((err - tol).max())
    assert kvr.device_status() == 0


@pytest.mark.parametrize("G", [3, 16])
def test_decode_shares_in_turns(G):
    """A line longer than the CTAs' greatest shares: each takes several.  64 sequences of 2^20 keys share their blocks."""
    gen = _gen(82)
    B, n, blocks = 64, 1 << 20, 64
    data = _tiles(gen, blocks * 64, 2.0 ** -9, torch.rand(blocks * 64, generator=gen, device=DEV).bfloat16().float()).view(blocks, 1, 64, -1)
    table = torch.zeros(n, 32, 2, device=DEV)
    table[..., 0] = 1.0
    bt = torch.arange(n // 1024, dtype=torch.int32, device=DEV) % blocks
    lens = torch.randint(1, n + 1, (B,), generator=gen, device=DEV)
    lens[0], lens[1], lens[2:] = n, 1, lens[2:].clamp(min=n // 2)
    pool = kvr.Kv8Layout(data, bt.repeat(B, 1).contiguous())
    q = torch.randn(B, G, 192, generator=gen, device=DEV).bfloat16()
    out = kvr.full_attn_decode_kv8(q, lens - 1, torch.arange(B, dtype=torch.int32, device=DEV), pool, table, SCALE, n)
    K, V = _values_gpu(data.view(-1, kvr.KV8_TILE))
    per = K.shape[0]
    for b in (0, 1, 2, 31, 63):
        m = int(lens[b])
        # every key appears m // per times, those of the first m % per once more
        times = torch.full((per,), float(m // per), dtype=torch.float64, device=DEV)
        times[:m % per] += 1
        s = q[b].double() @ K.T * SCALE
        w = torch.exp(s - s.amax(1, keepdim=True)) * times
        w = w / w.sum(1, keepdim=True)
        want, wv = w @ V, w @ V.abs()
        a = (q[b].double().abs() @ K.abs().T * SCALE).amax(1, keepdim=True)
        err = (out[b].double() - want).abs()
        tol = 2.0 ** -8 * want.abs() + (torch.exp(2 * 2.0 ** -10 * a) - 1) * (wv + want.abs()) + 2.0 ** -10 * wv
        assert torch.all(err <= tol), (b, float((err - tol).max()))
    assert kvr.device_status() == 0


@pytest.mark.parametrize("G", [8, 16])
def test_pool_past_4_gb(table, G):
    """Blocks whose bytes lie past 2^32, written, read and unpacked."""
    hkv, bs = 8, 1024
    nb = (9 << 29) // (hkv * (bs // 16) * kvr.KV8_TILE)   # 4.5 GB
    data = torch.empty(nb, hkv, bs // 16, kvr.KV8_TILE, dtype=torch.uint8, device=DEV)
    bt = _ints([[nb - 1, 0], [1, nb - 2]], torch.int32)
    pool = kvr.Kv8Layout(data, bt)
    gen = _gen(83)
    lens = [1100, 1030]
    k, v = _kv(gen, sum(lens), hkv)
    _append(pool, k, v, [0, 1], [0, 0], lens, table)
    q = torch.randn(2, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    small = kvr.Kv8Layout(data[[nb - 1, 0, 1, nb - 2]].contiguous(), _ints([[0, 1], [2, 3]], torch.int32))
    args = (q, _ints([1099, 1029], torch.int64), _ints([0, 1], torch.int32))
    out = kvr.full_attn_decode_kv8(*args, pool, table, SCALE, 1100)
    assert torch.equal(out, kvr.full_attn_decode_kv8(*args, small, table, SCALE, 1100))
    _check_decode(out, q, [1099, 1029], [0, 1], small, table)
    rows = kvr.LinearLayout.empty(sum(lens), hkv)
    kvr.kv8_unpack(pool, _ints([0, 1], torch.int32), _ints([0, 0], torch.int64), _ints([0, 1100, 2130], torch.int32), rows)
    wk, wv = _want_unpacked(small, 1, 0, 1030)
    assert torch.equal(rows.k[1100:].cpu(), wk) and torch.equal(rows.v[1100:].cpu(), wv)
    assert kvr.device_status() == 0


# -- unpack --------------------------------------------------------------------------------------------------------------

def _want_unpacked(pool, s, lo, n):
    data, bt = pool.data.cpu().numpy(), pool.block_table.cpu().numpy()
    ks, vs = [], []
    for h in range(pool.num_kv_heads):
        K, V, ok = o8.sequence(data, bt[s], h, lo + n)
        K[~ok], V[~ok] = 0, 0
        ks.append(torch.from_numpy(K[lo:].astype(np.float32)).bfloat16())  # (exact in fp32: one rounding)
        vs.append(torch.from_numpy(V[lo:].astype(np.float32)).bfloat16())
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
        kvr.kv8_unpack(pool, *args, dst)
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
        kvr.kv8_unpack(pool, *args, dst, dst_seqs=_ints(dseq, torch.int32), T=cu[-1])
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
    k, v = _kv(gen, 1, hkv)
    k[0, 1, 5], v[0, 0, 100] = float("nan"), float("inf")
    _append(pool, k, v, [0], [99], [1], table)
    rows = kvr.LinearLayout.empty(100, hkv)
    kvr.kv8_unpack(pool, _ints([0], torch.int32), _ints([0], torch.int64), _ints([0, 100], torch.int32), rows)
    wk, wv = torch.zeros(100, hkv, 192, dtype=torch.bool), torch.zeros(100, hkv, 128, dtype=torch.bool)
    wk[99, 1], wv[99, 0] = True, True                                       # a row that is not finite reads as NaN
    assert torch.equal(torch.isnan(rows.k).cpu(), wk) and torch.equal(torch.isnan(rows.v).cpu(), wv)
    pool.block_table[1, 1] = -1
    cu = [0, 50, 60, 70, 80, 90]
    dst = kvr.LinearLayout.empty(100, hkv)
    dst.k.fill_(9)
    kvr.kv8_unpack(pool, _ints([1, 2, -1, 0, 0], torch.int32), _ints([10, 0, 0, -5, 1 << 50], torch.int64),
                   _ints(cu, torch.int32), dst)
    assert kvr.device_status() == kvr.DEV_BAD_BLOCK | kvr.DEV_BAD_SEQ | kvr.DEV_BAD_POS
    k, _ = _want_unpacked(pool, 1, 10, 50)
    assert not k[22:].any() and torch.equal(dst.k[:50].cpu(), k)
    assert not dst.k[50:90].any() and (dst.k[90:] == 9).all()
    # row ranges that leave the call
    dst.k.fill_(9)
    for cu in ([40, 30], [90, 101], [-1, 30]):
        kvr.kv8_unpack(pool, _ints([0], torch.int32), _ints([0], torch.int64), _ints(cu, torch.int32), dst)
        assert kvr.device_status() == kvr.DEV_BAD_ROWS
    assert (dst.k == 9).all()
    # pages that cannot be addressed
    pages = kvr.PagedLayout.contiguous(2, hkv, 64, block_size=32)
    pages.k.fill_(9)
    pages.block_table[0, 1] = pages.num_blocks
    kvr.kv8_unpack(pool, _ints([0, 0], torch.int32), _ints([0, 0], torch.int64), _ints([0, 64, 90], torch.int32), pages,
                   dst_seqs=_ints([0, 2], torch.int32))
    assert kvr.device_status() == kvr.DEV_BAD_BLOCK | kvr.DEV_BAD_SEQ
    assert torch.equal(pages.k[0].transpose(0, 1).cpu(), _want_unpacked(pool, 0, 0, 32)[0]) and (pages.k[1:] == 9).all()


@pytest.mark.parametrize("hkv,S,mb", [(4, 3, 12), (1, 4096, 64)])
def test_unpack_into_a_wide_table(table, hkv, S, mb):
    """T left out: all that dst's table can name bounds the call, the rows there are decide it (past 65,536 CTAs it goes
    round), and rows at addresses that are 16-byte aligned only."""
    gen = _gen(mb)
    bs = 1024
    pool = _filled(gen, [700, 5], hkv, 64, table)
    base = torch.empty(3 * hkv * bs * 320 + 8, dtype=torch.bfloat16, device=DEV)[8:]
    base.fill_(9)
    k, v = base[:3 * hkv * bs * 192].view(3, hkv, bs, 192), base[3 * hkv * bs * 192:].view(3, hkv, bs, 128)
    bt = torch.full((S, mb), -1, dtype=torch.int32, device=DEV)
    bt[S - 1, 0], bt[0, 0] = 2, 1
    pages = kvr.PagedLayout(k, v, bt)
    kvr.kv8_unpack(pool, _ints([0, 1], torch.int32), _ints([0, 0], torch.int64), _ints([0, 700, 705], torch.int32), pages,
                   dst_seqs=_ints([S - 1, 0], torch.int32))
    assert kvr.device_status() == 0
    for blk, s, n in ((2, 0, 700), (1, 1, 5)):
        wk, wv = _want_unpacked(pool, s, 0, n)
        assert torch.equal(k[blk, :, :n].transpose(0, 1).cpu(), wk) and torch.equal(v[blk, :, :n].transpose(0, 1).cpu(), wv)
        assert (k[blk, :, n:] == 9).all()
    assert (k[0] == 9).all()
