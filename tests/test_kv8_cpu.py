"""The 8-bit pool and the calls on shared pages on the CPU: the oracle's scales,
codes and tile places against their definitions, its page bookkeeping against
hand-written cases and invariants, the library's host checks and the binding's
refusals."""
import ctypes

import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import kv8 as o8
from oracle import pages_share as ops
from sinks_kv_ring_gb300 import build as kbuild

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kvr.lib()


# -- the oracle ----------------------------------------------------------------------------------------------------------

def _is_bf16(s):
    return int(np.float32(s).view(np.uint32)) & 0xFFFF == 0


def test_least_scale():
    rng = np.random.default_rng(3)
    cases = np.concatenate([np.exp(rng.uniform(-80, 80, 3000)), 127.0 * 2.0 ** np.arange(-100, 100), [0, 1, 127, 1e-38, 1e-44, 3.3e38],
                            127.0 * (1 + np.arange(128) / 128), np.nextafter((127.0 * (1 + np.arange(128) / 128)).astype(np.float32), np.float32(1e9))])
    for a in cases.astype(np.float32):
        s = o8.least_scale(a)
        assert _is_bf16(s) and 127.0 * float(s) >= float(a)
        if s > 0:
            below = np.uint32(s.view(np.uint32) - 0x10000).view(np.float32)
            assert 127.0 * float(below) < float(a)
        assert (s == 0) == (a == 0)


def test_tile_places_cover_the_tile():
    at = np.concatenate([np.concatenate(o8.places(r)) for r in range(16)])
    assert np.array_equal(np.sort(at), np.arange(5120))


def test_codes_are_within_half_a_step():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((16, 192)) * np.exp(rng.uniform(-5, 5))).astype(np.float32)
    s = o8.least_scale(np.abs(x).max())
    u = o8.codes(x, s)
    assert np.abs(u).max() <= 127 and np.abs(u * float(s) - x).max() <= float(s) / 2 * (1 + 2.0 ** -20)
    assert np.array_equal(o8.codes(np.array([0.5, 1.5, -0.5, -2.5], np.float32), np.float32(1)), [0, 2, 0, -2])


def test_append_in_parts_keeps_what_is_there():
    """Chunks of a sequence written one after another: a value is off by half a step for each scale that it was held
    under, rows that are not finite read as NaN, and a tile's scale is its largest so far."""
    rng = np.random.default_rng(5)
    H, bs, n = 2, 32, 70
    data = rng.integers(0, 256, (5, H, bs // 16, o8.TILE)).astype(np.uint8)
    row = [3, 0, 4]
    k = rng.standard_normal((n, H, 192)).astype(np.float32) * np.exp(rng.uniform(-2, 2, (n, 1, 1))).astype(np.float32)
    v = rng.standard_normal((n, H, 128)).astype(np.float32)
    k[20, 1, 7], v[33, 0, 0] = np.nan, np.inf
    at = 0
    for c in (1, 1, 14, 5, 30, 2, 17):
        o8.append(data, row, at, k[at:at + c], v[at:at + c])
        at += c
    assert at == n
    for h in range(H):
        K, V, ok = o8.sequence(data, row, h, n)
        assert ok.all()
        for got, want, bad in ((K, k[:, h], (20, 1)), (V, v[:, h], (33, 0))):
            for p in range(n):
                if (p, h) == bad:
                    assert np.isnan(got[p]).all()
                    continue
                t = [q for q in range(p // 16 * 16, min(p // 16 * 16 + 16, n)) if (q, h) != bad]
                s = float(o8.least_scale(np.abs(want[t]).max()))
                assert np.abs(got[p] - want[p]).max() <= 8 * s  # at most 16 scales, each half a step of the last at most


def test_fork_free_and_compact_by_hand():
    t = np.array([[5, 2, 7, -1], [-1] * 4, [-1] * 4], np.int32)
    refs = np.zeros(9, np.int32)
    free = [0, 1, 3, 4, 6, 8]
    t1, r1, pairs, count, flags = ops.fork(t, 16, refs, [0, 0], [1, 2], [40, 32], free, 6)
    assert flags == 0 and count == 5 and pairs == [(7, 8)]
    assert t1.tolist() == [[5, 2, 7, -1], [5, 2, 8, -1], [5, 2, -1, -1]] and r1.tolist() == [0, 0, 2, 0, 0, 2, 0, 0, 0]
    assert ops.free(t1, 16, r1, [0, 1, 1], free, 5)[3:] == (5, ops.FREE_FULL)  # a list of six has no room for seven
    ids = free + [None] * 3
    t2, r2, ids, count, flags = ops.free(t1, 16, r1, [0, 1, 1], ids, 5)
    assert flags == 0 and count == 7 and ids[:7] == [0, 1, 3, 4, 6, 7, 8]
    assert (t2[:2] == -1).all() and r2.tolist() == [0] * 9
    t3, r3, left, pairs, flags = ops.compact(t2, r2, ids, 7)
    assert flags == 0 and pairs == [(2, 0), (5, 1)] and left == [8, 7, 6, 5, 4, 3, 2] and t3[2].tolist() == [1, 0, -1, -1]
    assert ops.compact(t2, r2, ids, 7, limit=1)[4] == ops.NO_BLOCKS
    # a part of a sequence: a window, and a cut
    t4, _, ids, count, _ = ops.free(t, 16, refs, [0], [None] * 9, 0, [20], [40])
    assert t4[0].tolist() == [-1, 2, 7, -1] and ids[:count] == [5]
    t4, _, ids, count, _ = ops.free(t, 16, refs, [0], [None] * 9, 0, None, [17])
    assert t4[0].tolist() == [5, 2, -1, -1] and ids[:count] == [7]


def test_page_bookkeeping_keeps_every_block():
    """Random forks, frees and compactions: at every moment each block is either free or held by refs + 1 entries."""
    rng = np.random.default_rng(6)
    S, mb, bs, nb = 12, 6, 16, 40
    t, refs = np.full((S, mb), -1, np.int32), np.zeros(nb, np.int32)
    free, count = list(rng.permutation(nb)), nb
    lens = [0] * S
    for step in range(300):
        what = rng.integers(4)
        if what == 0:  # a new request
            s = int(rng.integers(S))
            need = int(rng.integers(1, mb + 1))
            if lens[s] == 0 and count >= need:
                for j in range(need):
                    count -= 1
                    t[s, j] = free[count]
                lens[s] = int(rng.integers((need - 1) * bs + 1, need * bs + 1))
        elif what == 1:
            live, idle = [s for s in range(S) if lens[s]], [s for s in range(S) if not lens[s]]
            if live and idle:
                src = [int(rng.choice(live)) for _ in idle[:3]]
                n = [int(rng.integers(0, lens[s] + 1)) for s in src]
                t, refs, pairs, count, flags = ops.fork(t, bs, refs, src, idle[:3], n, free, count)
                if flags == 0:
                    for d, m in zip(idle[:3], n):
                        lens[d] = m
        elif what == 2:
            s = [int(x) for x in rng.permutation(S)[:4]]
            keep = [int(rng.integers(0, max(lens[x], 1))) for x in s]
            t, refs, free, count, flags = ops.free(t, bs, refs, s, free, count, None, keep)
            for x, m in zip(s, keep):
                lens[x] = min(lens[x], m)
        elif count > 0:
            t, refs, left, pairs, flags = ops.compact(t, refs, free, count)
            free = left + free[count:]
            assert flags == 0 and count == len(left)
        holders = np.bincount(t[t >= 0], minlength=nb)
        gone = set(free[:count])
        assert len(gone) == count
        for b in range(nb):
            assert (b in gone and holders[b] == 0 and refs[b] == 0) or (b not in gone and holders[b] == refs[b] + 1)


# -- host validation -----------------------------------------------------------------------------------------------------

def _pool(**kw):
    d = dict(num_kv_heads=4, num_seqs=4, max_blocks=16, block_size=64, num_blocks=64, data=FAKE, block_table=FAKE)
    d.update(kw)
    return kvr._Layout4(**d)


def test_kv8_host_validation_codes(L):
    P, odd = ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 2)
    R = ctypes.byref

    def app(k=P, v=P, cu=P, P0=P, seqs=P, n=3, T=8, H=4, table=P, max_pos=1000, dst=_pool()):
        return L.kv8_append_rope(k, v, cu, P0, seqs, n, T, H, table, max_pos, 0.7, R(dst) if dst else None, None)

    assert app(n=-1) == -1 and app(T=-1) == -1 and app(T=1 << 31) == -1 and app(H=2) == -1 and app(dst=None) == -1
    for name in ("k", "v", "cu", "P0", "seqs", "table"):
        assert app(**{name: None}) == -1, name
    assert app(k=odd) == -1 and app(v=odd) == -1 and app(table=odd) == -1
    assert app(max_pos=0) == -2 and app(dst=_pool(data=FAKE + 8)) == -1 and app(dst=_pool(block_table=None)) == -1
    assert app(dst=_pool(block_size=40)) == -4 and app(dst=_pool(block_size=2048)) == -4
    assert app(dst=_pool(max_blocks=(1 << 25) + 1, block_size=1024)) == -4
    assert app(k=None, v=None, n=0) == 0 and app(k=None, v=None, T=0) == 0

    dec, size = L.full_attn_decode_kv8, L.full_attn_decode_kv8_workspace_size
    need = size(2, 64, 4, 10000)
    assert need > 0 and size(2, 62, 4, 10000) == 0 and size(0, 64, 4, 10000) == 0 and size(2, 64, 4, 0) == 0
    assert size(2, 64, 4, 1000) == 0                                                  # short contexts need none
    pool, long = _pool(), _pool(max_blocks=200)
    assert dec(P, P, P, 2, 64, R(long), P, 10000, 0.1, 10000, P, need - 1, P, None) == -3
    assert dec(P, P, P, 2, 64, R(long), P, 10000, 0.1, 10000, None, need, P, None) == -3
    assert dec(P, P, P, 2, 64, R(pool), P, 1000, 0.1, 1001, P, 1 << 40, P, None) == -2
    assert dec(P, P, P, 2, 64, R(pool), P, 5000, 0.1, 1025, P, 1 << 40, P, None) == -2
    assert dec(P, P, P, 2, 62, R(pool), P, 1000, 0.1, 100, P, 1 << 40, P, None) == -1
    assert dec(P, P, P, 2, 128, R(pool), P, 1000, 0.1, 100, P, 1 << 40, P, None) == -4   # 32 heads per KV head
    assert dec(P, P, P, 2, 64, R(pool), P, 1000, 0.1, 100, P, 1 << 40, odd, None) == -1
    assert dec(P, P, P, 2, 64, R(pool), P, 1000, 0.1, 100, ctypes.c_void_p(FAKE + 8), 1 << 40, P, None) == -1
    huge = _pool(max_blocks=1 << 25)
    assert dec(P, P, P, 2, 64, R(huge), P, (1 << 31) - 1, 0.1, (1 << 30) + 1, P, 1 << 62, P, None) == -4
    assert dec(None, None, None, 0, 64, R(pool), P, 1000, 0.1, 100, None, 0, None, None) == 0

    unp = L.kv8_unpack
    lin = kvr._Layout(kind=3, num_kv_heads=4, k=FAKE, v=FAKE, num_rows=100)
    ring = kvr._Layout(kind=1, num_kv_heads=4, k=FAKE, v=FAKE, slot_pos=FAKE, num_seqs=4)
    pages = kvr._Layout(kind=2, num_kv_heads=4, k=FAKE, v=FAKE, block_table=FAKE, num_seqs=4, max_blocks=16,
                        block_size=64, num_blocks=64)
    assert unp(R(pool), P, P, P, 1, 10, None, R(ring), None) == -1
    assert unp(R(_pool(num_kv_heads=2)), P, P, P, 1, 10, None, R(lin), None) == -1
    assert unp(R(pool), P, P, P, 1, 101, None, R(lin), None) == -1                    # more rows than dst has
    assert unp(R(pool), P, P, P, 1, 10, None, R(pages), None) == -1                   # no dst_seqs
    assert unp(R(pool), None, P, P, 1, 10, None, R(lin), None) == -1
    assert unp(R(pool), P, P, P, -1, 10, None, R(lin), None) == -1
    assert unp(R(pool), P, P, P, 0, 10, None, R(lin), None) == 0
    assert unp(R(pool), P, P, P, 3, 0, None, R(lin), None) == 0


def test_shared_pages_host_validation_codes(L):
    P = ctypes.c_void_p(FAKE)

    def free(table=P, S=4, mb=16, bs=64, nb=64, refs=P, seqs=P, klo=None, khi=None, n=1, ids=P, count=P, cap=8):
        return L.kv_pages_free(table, S, mb, bs, nb, refs, seqs, klo, khi, n, ids, count, cap, None)

    def fork(table=P, S=4, mb=16, bs=64, nb=64, refs=P, src=P, dst=P, lens=P, n=1, ids=P, cin=P, cout=P, cap=8, a=P, b=P,
             c=P):
        return L.kv_pages_fork(table, S, mb, bs, nb, refs, src, dst, lens, n, ids, cin, cout, cap, a, b, c, None)

    def comp(table=P, tout=P, S=4, mb=16, nb=64, limit=0, refs=P, rout=P, ids=P, count=P, iout=P, cap=8, a=P, b=P, c=P):
        return L.kv_pages_compact(table, tout, S, mb, nb, limit, refs, rout, ids, count, iout, cap, a, b, c, None)

    for call in (free, fork, comp):
        assert call(S=0) == -1 and call(mb=0) == -1 and call(nb=0) == -1 and call(cap=-1) == -1 and call(nb=(1 << 30) + 1) == -4
        for k in ("table", "refs", "ids"):
            assert call(**{k: None}) == -1, k
    assert free(bs=0) == -1 and free(n=-1) == -1 and free(seqs=None) == -1 and free(count=None) == -1
    assert free(klo=P) == -1                                                          # a lower bound alone
    assert free(n=0, seqs=None) == 0
    assert fork(bs=0) == -1 and fork(n=-1) == -1 and fork(n=8193) == -4
    for k in ("src", "dst", "lens", "cin", "cout", "a", "b", "c"):
        assert fork(**{k: None}) == -1, k
    for k in ("tout", "rout", "count", "iout", "a", "b", "c"):
        assert comp(**{k: None}) == -1, k
    assert comp(limit=-1) == -1 and comp(nb=(1 << 20) + 1) == -4

    def copy(planes=(FAKE,), sizes=(64,), nb=8, a=P, b=P, c=P, n=3):
        pl = (ctypes.c_void_p * len(planes))(*planes) if planes else None
        sz = (ctypes.c_int64 * len(sizes))(*sizes) if sizes else None
        return L.kv_pages_copy(pl, sz, max(len(planes), len(sizes)), nb, a, b, c, n, None)

    assert copy(planes=()) == -1 and copy(sizes=()) == -1 and copy(planes=(None,)) == -1 and copy(planes=(FAKE + 8,)) == -1
    assert copy(sizes=(40,)) == -1 and copy(sizes=(0,)) == -1 and copy(nb=0) == -1 and copy(n=-1) == -1
    assert copy(a=None) == -1 and copy(b=None) == -1 and copy(c=None) == -1
    assert copy(n=0) == 0 and copy(planes=(), sizes=()) == 0


# -- the binding ---------------------------------------------------------------------------------------------------------

class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("workspace_size") else 0
        return call


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    want = kvr._want
    monkeypatch.setattr(kvr, "lib", lambda: r)
    monkeypatch.setattr(kvr, "_want", lambda t, name, dtype, dim=None, cuda=True: want(t, name, dtype, dim, cuda=False))
    monkeypatch.setattr(kvr, "_stream", lambda s: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    return r


def _z(dtype, *shape):
    return torch.zeros(*shape, dtype=dtype)


BF, I32, I64, F32, U8 = torch.bfloat16, torch.int32, torch.int64, torch.float32, torch.uint8


def _page_args(nb=12):
    return dict(table=_z(I32, 3, 4), refs=_z(I32, nb), ids=_z(I32, nb), count=_z(I32, 1), a=_z(I32, nb), b=_z(I32, nb), c=_z(I32, 1))


def test_good_calls_reach_the_library(rec):
    pool = kvr.Kv8Layout.contiguous(3, 2, 100, block_size=32, device="cpu")
    assert (pool.block_size, pool.max_blocks, pool.num_blocks) == (32, 4, 12) and kvr.Kv8Layout.bytes_per_token(4) == 1284
    table = _z(F32, 300, 32, 2)
    kvr.kv8_append_rope(_z(BF, 5, 2, 192), _z(BF, 5, 2, 128), _z(I32, 3), _z(I64, 2), _z(I32, 2), table, 0.7, pool)
    out = kvr.full_attn_decode_kv8(_z(BF, 3, 16, 192), _z(I64, 3), _z(I32, 3), pool, table, 0.1, 100)
    assert tuple(out.shape) == (3, 16, 128)
    kvr.kv8_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3), kvr.LinearLayout.empty(9, 2, device="cpu"))
    pages = kvr.PagedLayout.contiguous(3, 2, 100, block_size=32, device="cpu")
    kvr.kv8_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3), pages, dst_seqs=_z(I32, 2), T=70)
    x = _page_args()
    kvr.kv_pages_free(x["table"], 12, 32, x["refs"], _z(I32, 2), x["ids"], x["count"], keep_hi=_z(I64, 2))
    kvr.kv_pages_fork(x["table"], 12, 32, x["refs"], _z(I32, 2), _z(I32, 2), _z(I64, 2), x["ids"], x["count"], x["a"], x["b"], x["c"])
    kvr.kv_pages_compact(x["table"], 12, x["refs"], x["ids"], x["count"], x["a"][:6].contiguous(), x["b"], x["c"], limit=9,
                         refs_out=_z(I32, 12))
    kvr.kv_pages_copy([pool, pages, kvr.Kv4Layout.contiguous(3, 2, 100, block_size=32, device="cpu")], x["a"], x["b"], x["c"])
    kvr.kv_pages_copy(pool, x["a"], x["b"], x["c"])
    kvr.kv_pages_copy([], x["a"], x["b"], x["c"])
    calls = [(n, a) for n, a in rec.calls if not n.endswith("workspace_size")]
    assert [n for n, _ in calls] == ["kv8_append_rope", "full_attn_decode_kv8", "kv8_unpack", "kv8_unpack", "kv_pages_free",
                                     "kv_pages_fork", "kv_pages_compact", "kv_pages_copy", "kv_pages_copy"]
    assert [a[5] for n, a in calls if n == "kv8_unpack"] == [9, 70]
    planes, sizes, n = calls[7][1][:3]
    assert n == 4 and list(sizes) == [2 * 2 * 5136, 2 * 32 * 384, 2 * 32 * 256, 2 * 2 * 2912]


def test_copy_of_a_pool_of_one_block_cut_out_of_others(rec):
    """The stride of an axis of one says nothing: the block is as large as its tensor."""
    data = _z(U8, 5, 2, 2, 5136)[::5]
    assert data.is_contiguous() and data.stride(0) == 5 * 2 * 2 * 5136
    x = _page_args()
    kvr.kv_pages_copy(kvr.Kv8Layout(data, _z(I32, 3, 4)), x["a"], x["b"], x["c"])
    assert list(rec.calls[-1][1][1]) == [2 * 2 * 5136]


def test_binding_refuses_before_the_library(rec):
    pool = kvr.Kv8Layout.contiguous(3, 2, 100, block_size=32, device="cpu")
    pool4 = kvr.Kv4Layout.contiguous(3, 2, 100, block_size=32, device="cpu")
    lin = kvr.LinearLayout.empty(9, 2, device="cpu")
    table = _z(F32, 300, 32, 2)
    k, v, cu, P0, seqs = _z(BF, 5, 2, 192), _z(BF, 5, 2, 128), _z(I32, 3), _z(I64, 2), _z(I32, 2)
    q, pos, seq = _z(BF, 3, 16, 192), _z(I64, 3), _z(I32, 3)
    x = _page_args()
    t, refs, ids, count, a, b, c = (x[n] for n in ("table", "refs", "ids", "count", "a", "b", "c"))
    bad = [
        lambda: kvr.Kv8Layout(_z(U8, 2, 2, 4, 5120), _z(I32, 1, 2)),
        lambda: kvr.Kv8Layout(_z(torch.int8, 2, 2, 4, 5136), _z(I32, 1, 2)),
        lambda: kvr.Kv8Layout.contiguous(2, 2, 100, block_size=24, device="cpu"),
        lambda: kvr.kv8_append_rope(k, v, cu, P0, seqs, table, 0.7, pool4),
        lambda: kvr.kv8_append_rope(k, v, cu[:2].contiguous(), P0, seqs, table, 0.7, pool),
        lambda: kvr.kv8_append_rope(k, v, cu, _z(I64, 3), seqs, table, 0.7, pool),
        lambda: kvr.kv8_append_rope(k, v[:4].contiguous(), cu, P0, seqs, table, 0.7, pool),
        lambda: kvr.kv8_append_rope(k.transpose(0, 1), v, cu, P0, seqs, table, 0.7, pool),
        lambda: kvr.kv8_append_rope(k.float(), v, cu, P0, seqs, table, 0.7, pool),
        lambda: kvr.kv8_append_rope(k, v, cu, P0.int(), seqs, table, 0.7, pool),
        lambda: kvr.full_attn_decode_kv8(q, pos, seq, pool4, table, 0.1, 100),
        lambda: kvr.full_attn_decode_kv4(q, pos, seq, pool, table, 0.1, 100),
        lambda: kvr.full_attn_decode_kv8(q[..., :128].contiguous(), pos, seq, pool, table, 0.1, 100),
        lambda: kvr.full_attn_decode_kv8(q, _z(I64, 2), seq, pool, table, 0.1, 100),
        lambda: kvr.full_attn_decode_kv8(q, pos, seq, pool, table, 0.1, 100, out=_z(BF, 3, 16, 192)),
        lambda: kvr.kv8_unpack(pool4, seqs, P0, cu, lin),
        lambda: kvr.kv8_unpack(pool, seqs, P0, cu[:2].contiguous(), lin),
        lambda: kvr.kv8_unpack(pool, seqs, P0, cu, kvr.PagedLayout.contiguous(2, 2, 100, device="cpu")),
        lambda: kvr.kv8_unpack(pool, seqs, P0, cu, kvr.RingLayout.empty(1, 2, device="cpu")),
        lambda: kvr.kv_pages_free(t, 13, 32, refs, seqs, ids, count),
        lambda: kvr.kv_pages_free(t, 12, 32, refs.long(), seqs, ids, count),
        lambda: kvr.kv_pages_free(t, 12, 32, refs, seqs, ids, _z(I32, 2)),
        lambda: kvr.kv_pages_free(t, 12, 32, refs, seqs, ids, count, keep_hi=_z(I64, 3)),
        lambda: kvr.kv_pages_free(t, 12, 32, refs, seqs, ids, count, keep_lo=_z(I32, 2), keep_hi=_z(I64, 2)),
        lambda: kvr.kv_pages_fork(t, 12, 32, refs, seqs, _z(I32, 3), P0, ids, count, a, b, c),
        lambda: kvr.kv_pages_fork(t, 12, 32, refs, seqs, seqs, _z(I64, 1), ids, count, a, b, c),
        lambda: kvr.kv_pages_fork(t, 12, 32, refs, seqs, seqs, P0, ids, count, _z(I32, 1), b, c),
        lambda: kvr.kv_pages_fork(t, 12, 32, refs, seqs, seqs, P0, ids, count, a, b, _z(I32, 2)),
        lambda: kvr.kv_pages_fork(t, 12, 32, refs[:11].contiguous(), seqs, seqs, P0, ids, count, a, b, c),
        lambda: kvr.kv_pages_compact(t, 12, refs, ids, count, _z(I32, 5), b, c),
        lambda: kvr.kv_pages_compact(t, 12, refs, ids, count, a, b, c, table_out=_z(I32, 3, 5)),
        lambda: kvr.kv_pages_compact(t, 12, refs, ids, count, a, b, c, refs_out=_z(I64, 12)),
        lambda: kvr.kv_pages_copy([pool, lin], a, b, c),
        lambda: kvr.kv_pages_copy([pool, kvr.Kv8Layout.contiguous(2, 2, 100, block_size=32, device="cpu")], a, b, c),
        lambda: kvr.kv_pages_copy(pool, a.long(), b, c),
        lambda: kvr.kv_pages_copy(pool, a, b, _z(I32, 2)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"case {i} was taken")
    assert [n for n, _ in rec.calls if not n.endswith("workspace_size")] == []
