"""The 4-bit pool and page growth without a GPU: the oracle against worked
examples and its own invariants, host validation of the C calls, refusals of
the binding."""
import ctypes

import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import kv4 as o4
from sinks_kv_ring_gb300 import build as kbuild

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kvr.lib()


# -- the oracle itself ---------------------------------------------------------------------------------------------------

def test_every_byte_of_a_tile_has_one_owner():
    seen = {}
    for r in range(16):
        kc, vc, *halves = o4.places(r)
        own = set(kc) | set(vc) | {a + b for at in halves for a in at for b in (0, 1)} | {2790 + 8 * r, 2791 + 8 * r}
        assert len(own) == 96 + 64 + 2 * (3 + 2 + 2 + 3) + 2
        for b in own:
            assert b not in seen, (r, b, seen[b])
            seen[b] = r
        # a code byte holds two neighbouring dims of the position
        assert all(kc[2 * i] == kc[2 * i + 1] for i in range(96)) and all(vc[2 * i] == vc[2 * i + 1] for i in range(64))
    assert sorted(seen) == list(range(o4.TILE))


def test_write_then_read_gives_the_dequantised_values():
    rng = np.random.default_rng(3)
    data = np.full((2, 3, 2, o4.TILE), 0xFF, np.uint8)
    for row in range(32):
        k, v = rng.standard_normal(192).astype(np.float32), rng.standard_normal(128).astype(np.float32) * 3
        kq, vq = o4.quantise(k), o4.quantise(v)
        o4.write(data, 1, 2, row, *kq, *vq)
        K, V = o4.read(data[1, 2, row // 16])
        assert np.array_equal(K[row % 16], o4.dequantise(*kq)) and np.array_equal(V[row % 16], o4.dequantise(*vq))


def test_quantiser_error_is_half_a_step_and_the_ends_are_held():
    rng = np.random.default_rng(4)
    for scale in (1e-3, 1.0, 300.0):
        for off in (0.0, 5.0, -40.0):
            x = (rng.standard_normal((200, 128)) * scale + off).astype(np.float32)
            u, s, m = o4.quantise(x)
            y = o4.dequantise(u, s, m)
            step = np.repeat(s.astype(np.float64), 64, -1).reshape(x.shape)
            # half a step, and the fp32 rounding of x - m and of the quotient (16 units of 2^-24)
            assert np.all(np.abs(y - x) <= step * (0.5 + 16 * 2.0 ** -24) + np.abs(x) * 2.0 ** -24)
            g = x.reshape(200, 2, 64)
            assert np.all(m <= g.min(-1))
            # max x - m and its fifteenth are each rounded by 2^-24 of max x - m <= 2.01 max |x|
            assert np.all(m.astype(np.float64) + 15 * s.astype(np.float64) >= g.max(-1) - 2.0 ** -22 * np.abs(g).max(-1))


def test_quantiser_corner_groups():
    one = np.ones(64, np.float32)
    u, s, m = o4.quantise(one * 3)           # a constant that fp16 holds: no step
    assert not u.any() and s == 0 and m == 3
    u, s, m = o4.quantise(one * np.float32(0.1))
    assert abs(o4.dequantise(u, s, m) - 0.1).max() <= float(s[0]) / 2 + 1e-9
    x = one.copy()
    x[5] = np.nan
    u, s, m = o4.quantise(x)
    assert not u.any() and np.isnan(s) and np.isnan(m)
    u, s, m = o4.quantise(np.linspace(-1e30, 1e30, 64).astype(np.float32))
    assert m == -65504 and s == 65504 and u.min() == 0 and u.max() == 15
    u, s, m = o4.quantise(np.linspace(0, 1e-9, 64).astype(np.float32))  # below fp16's least step
    assert m == 0 and float(s[0]) == 2.0 ** -24


def test_ties_round_to_even():
    x = np.zeros(64, np.float32)
    x[1], x[2], x[3], x[4] = 15, 0.5, 1.5, 2.5  # m = 0, s = 1
    u, s, m = o4.quantise(x)
    assert (s, m) == (1, 0) and u[1:5].tolist() == [15, 0, 2, 2]


def test_grow_worked_example():
    table = np.full((3, 4), -1, np.int32)
    table[2, 0], table[0, :2] = 7, (1, 5)
    free = np.array([9, 8, 6, 4], np.int32)
    t, c, cu, pos, rseq, slots, fl = o4.grow(table, 16, 10, [2, 0], [15, 32], [2, 1], free, 4, 5)
    assert (c, fl) == (2, 0) and cu.tolist() == [0, 2, 3]
    assert t[2].tolist() == [7, 4, -1, -1] and t[0].tolist() == [1, 5, 6, -1]
    assert pos.tolist() == [15, 16, 32, -1, -1] and rseq.tolist() == [2, 2, 0, -1, -1]
    assert slots.tolist() == [7 * 16 + 15, 4 * 16, 6 * 16, -1, -1]


# -- host validation -----------------------------------------------------------------------------------------------------

def _pool(**kw):
    d = dict(num_kv_heads=4, num_seqs=4, max_blocks=16, block_size=64, num_blocks=64, data=FAKE, block_table=FAKE)
    d.update(kw)
    return kvr._Layout4(**d)


def test_kv4_host_validation_codes(L):
    P = ctypes.c_void_p(FAKE)
    R = ctypes.byref
    pool = _pool()
    app = L.kv4_append_rope
    assert app(P, P, P, P, None, -1, 4, P, 1000, 0.7, R(pool), None) == -1
    assert app(P, P, P, P, None, 8, 2, P, 1000, 0.7, R(pool), None) == -1            # Hkv
    assert app(P, P, P, P, P, 8, 4, P, 1000, 0.7, R(pool), None) == -1               # both seq and slots
    assert app(P, P, P, None, None, 8, 4, P, 1000, 0.7, R(pool), None) == -1         # neither
    assert app(ctypes.c_void_p(FAKE + 2), P, P, P, None, 8, 4, P, 1000, 0.7, R(pool), None) == -1
    assert app(P, P, P, P, None, 8, 4, P, 1000, 0.7, None, None) == -1
    assert app(P, P, P, P, None, 8, 4, P, 1000, 0.7, R(_pool(data=FAKE + 8)), None) == -1
    assert app(P, P, P, P, None, 8, 4, P, 1000, 0.7, R(_pool(block_table=None)), None) == -1
    assert app(P, P, P, P, None, 8, 4, P, 1000, 0.7, R(_pool(block_size=40)), None) == -4
    assert app(P, P, P, P, None, 8, 4, P, 1000, 0.7, R(_pool(block_size=2048)), None) == -4
    far = _pool(max_blocks=(1 << 25) + 1, block_size=1024)                            # past 2^35 positions a sequence
    assert app(P, P, P, P, None, 8, 4, P, 1000, 0.7, R(far), None) == -4
    assert app(P, P, P, P, None, 8, 4, P, 0, 0.7, R(pool), None) == -2
    assert app(None, None, None, None, None, 0, 4, P, 1000, 0.7, R(pool), None) == 0

    dec, size = L.full_attn_decode_kv4, L.full_attn_decode_kv4_workspace_size
    need = size(2, 64, 4, 10000)
    assert need > 0 and size(2, 62, 4, 10000) == 0 and size(0, 64, 4, 10000) == 0 and size(2, 64, 4, 0) == 0
    assert size(2, 64, 4, 1000) == 0                                                  # short contexts need none
    long = _pool(max_blocks=200)
    assert dec(P, P, P, 2, 64, R(long), P, 10000, 0.1, 10000, P, need - 1, P, None) == -3
    assert dec(P, P, P, 2, 64, R(long), P, 10000, 0.1, 10000, None, need, P, None) == -3
    assert dec(P, P, P, 2, 64, R(pool), P, 1000, 0.1, 1001, P, 1 << 40, P, None) == -2
    assert dec(P, P, P, 2, 64, R(pool), P, 5000, 0.1, 1025, P, 1 << 40, P, None) == -2
    assert dec(P, P, P, 2, 62, R(pool), P, 1000, 0.1, 100, P, 1 << 40, P, None) == -1
    assert dec(P, P, P, 2, 128, R(pool), P, 1000, 0.1, 100, P, 1 << 40, P, None) == -4   # 32 heads per KV head
    assert dec(P, P, P, 2, 64, R(pool), P, 1000, 0.1, 100, P, 1 << 40, ctypes.c_void_p(FAKE + 2), None) == -1
    assert dec(P, P, P, 2, 64, R(pool), P, 1000, 0.1, 100, ctypes.c_void_p(FAKE + 8), 1 << 40, P, None) == -1
    assert dec(None, None, None, 0, 64, R(pool), P, 1000, 0.1, 100, None, 0, None, None) == 0

    unp = L.kv4_unpack
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


def test_grow_host_validation_codes(L):
    P = ctypes.c_void_p(FAKE)
    grow = L.kv_pages_grow

    def call(table=P, S=4, mb=16, bs=64, nb=64, seqs=P, lens=P, add=P, n=1, ids=P, cin=P, cout=P, cap=8, cu=P, pos=P,
             rs=P, sl=P, T=8):
        return grow(table, S, mb, bs, nb, seqs, lens, add, n, ids, cin, cout, cap, cu, pos, rs, sl, T, None)

    assert call(n=-1) == -1 and call(T=-1) == -1 and call(T=1 << 31) == -1 and call(cap=-1) == -1
    assert call(S=0) == -1 and call(mb=0) == -1 and call(bs=0) == -1 and call(nb=0) == -1
    for k in ("table", "seqs", "lens", "add", "ids", "cin", "cout", "cu", "pos", "rs", "sl"):
        assert call(**{k: None}) == -1, k
    assert call(n=8193) == -4


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


BF, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


def test_layout_shapes():
    pool = kvr.Kv4Layout.__new__(kvr.Kv4Layout)
    assert kvr.Kv4Layout.bytes_per_token(4) == 728 and pool is not None
    with pytest.raises(ValueError):
        kvr.Kv4Layout.contiguous(2, 2, 100, block_size=24, device="cpu")


def test_good_calls_reach_the_library(rec):
    pool = kvr.Kv4Layout.contiguous(3, 2, 100, block_size=32, device="cpu")
    assert (pool.block_size, pool.max_blocks, pool.num_blocks) == (32, 4, 12)
    table = _z(F32, 300, 32, 2)
    kvr.kv4_append_rope(_z(BF, 5, 2, 192), _z(BF, 5, 2, 128), _z(I64, 5), _z(I32, 5), table, 0.7, pool)
    kvr.kv4_append_rope(_z(BF, 5, 2, 192), _z(BF, 5, 2, 128), _z(I64, 5), None, table, 0.7, pool, slots=_z(I64, 5))
    out = kvr.full_attn_decode_kv4(_z(BF, 3, 16, 192), _z(I64, 3), _z(I32, 3), pool, table, 0.1, 100)
    assert tuple(out.shape) == (3, 16, 128)
    kvr.kv4_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3), kvr.LinearLayout.empty(9, 2, device="cpu"))
    pages = kvr.PagedLayout.contiguous(2, 2, 100, block_size=64, device="cpu")
    kvr.kv4_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3), pages, dst_seqs=_z(I32, 2), T=70)
    kvr.kv_pages_grow(_z(I32, 3, 4), 12, 32, _z(I32, 2), _z(I64, 2), _z(I32, 2), _z(I32, 12), _z(I32, 1), _z(I32, 3),
                      _z(I64, 6), _z(I32, 6), _z(I64, 6))
    names = [n for n, _ in rec.calls if not n.endswith("workspace_size")]
    assert names == ["kv4_append_rope", "kv4_append_rope", "full_attn_decode_kv4", "kv4_unpack", "kv4_unpack",
                     "kv_pages_grow"]
    assert [a[5] for n, a in rec.calls if n == "kv4_unpack"] == [9, 70]


def test_binding_refuses_before_the_library(rec):
    pool = kvr.Kv4Layout.contiguous(3, 2, 100, block_size=32, device="cpu")
    table = _z(F32, 300, 32, 2)
    k, v, pos, seq, sl = _z(BF, 5, 2, 192), _z(BF, 5, 2, 128), _z(I64, 5), _z(I32, 5), _z(I64, 5)
    bad = [
        lambda: kvr.Kv4Layout(_z(torch.uint8, 2, 2, 4, 2880), _z(I32, 1, 2)),
        lambda: kvr.Kv4Layout(_z(torch.int8, 2, 2, 4, 2912), _z(I32, 1, 2)),
        lambda: kvr.kv4_append_rope(k, v, pos, None, table, 0.7, pool),
        lambda: kvr.kv4_append_rope(k, v, pos, seq, table, 0.7, pool, slots=sl),
        lambda: kvr.kv4_append_rope(k, v, pos, seq[:4].contiguous(), table, 0.7, pool),
        lambda: kvr.kv4_append_rope(k, v, pos, None, table, 0.7, pool, slots=sl[:4].contiguous()),
        lambda: kvr.kv4_append_rope(k, v[:4].contiguous(), pos, seq, table, 0.7, pool),
        lambda: kvr.kv4_append_rope(k.transpose(0, 1), v, pos, seq, table, 0.7, pool),
        lambda: kvr.kv4_append_rope(k.float(), v, pos, seq, table, 0.7, pool),
        lambda: kvr.full_attn_decode_kv4(_z(BF, 3, 16, 128), _z(I64, 3), _z(I32, 3), pool, table, 0.1, 100),
        lambda: kvr.full_attn_decode_kv4(_z(BF, 3, 16, 192), _z(I64, 2), _z(I32, 3), pool, table, 0.1, 100),
        lambda: kvr.full_attn_decode_kv4(_z(BF, 3, 16, 192), _z(I64, 3), _z(I32, 3), pool, table, 0.1, 100,
                                         out=_z(BF, 3, 16, 192)),
        lambda: kvr.kv4_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 2), kvr.LinearLayout.empty(9, 2, device="cpu")),
        lambda: kvr.kv4_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3),
                               kvr.PagedLayout.contiguous(2, 2, 100, device="cpu")),
        lambda: kvr.kv4_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3), kvr.RingLayout.empty(1, 2, device="cpu")),
        lambda: kvr.kv_pages_grow(_z(I32, 3, 4), 12, 32, _z(I32, 2), _z(I64, 2), _z(I32, 2), _z(I32, 12), _z(I32, 1),
                                  _z(I32, 2), _z(I64, 6), _z(I32, 6), _z(I64, 6)),
        lambda: kvr.kv_pages_grow(_z(I32, 3, 4), 12, 32, _z(I32, 2), _z(I64, 2), _z(I64, 2), _z(I32, 12), _z(I32, 1),
                                  _z(I32, 3), _z(I64, 6), _z(I32, 6), _z(I64, 6)),
        lambda: kvr.kv_pages_grow(_z(I32, 3, 4), 12, 32, _z(I32, 2), _z(I64, 2), _z(I32, 2), _z(I32, 12), _z(I32, 1),
                                  _z(I32, 3), _z(I64, 6), _z(I32, 5), _z(I64, 6)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail(f"case {i} was taken")
    assert [n for n, _ in rec.calls if not n.endswith("workspace_size")] == []
