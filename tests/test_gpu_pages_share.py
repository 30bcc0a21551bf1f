"""Shared pages on the GPU: giving blocks up, forking, compacting and the block
copies, each against plain Python; and a run of them with the calls they stand
beside, over pools in bf16, 4 and 8 bits."""
import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import pages_share as ops

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


def _t(v, t=torch.int32):
    return torch.tensor(np.asarray(v).tolist(), dtype=t, device=DEV)


def _state(rng, S, mb, bs, nb, shared=0.5):
    """Tables of some sequences, a part of them forked from others; the free list; everybody's lengths."""
    table, refs = np.full((S, mb), -1, np.int32), np.zeros(nb, np.int32)
    free, count = rng.permutation(nb).astype(np.int32), nb
    lens = np.zeros(S, np.int64)
    for s in rng.permutation(S)[:max(1, S // 2)]:
        need = int(rng.integers(0, min(mb, max(count // 4, 1)) + 1))
        for j in range(need):
            count -= 1
            table[s, j] = free[count]
        lens[s] = max(need * bs - int(rng.integers(0, bs)), 0)
    live, idle = np.nonzero(lens)[0], np.nonzero(lens == 0)[0]
    if len(live) and shared:
        dst = idle[rng.random(len(idle)) < shared]
        src = rng.choice(live, len(dst))
        n = [int(rng.integers(0, lens[s] + 1)) for s in src]
        table, refs, _, count, flags = ops.fork(table, bs, refs, src, dst, n, free, count)
        if flags == 0:
            lens[dst] = n
    return table, refs, free, count, lens


# -- free ----------------------------------------------------------------------------------------------------------------

def _free(table, bs, nb, refs, seqs, free, count, lo=None, hi=None):
    t, r, ids, c = _t(table), _t(refs), _t(free), _t([count])
    kvr.kv_pages_free(t, nb, bs, r, _t(seqs), ids, c, None if lo is None else _t(lo, torch.int64),
                      None if hi is None else _t(hi, torch.int64))
    flags = kvr.device_status()
    wt, wr, wids, wc, wf = ops.free(table, bs, refs, seqs, free, count, lo, hi)
    assert flags == wf
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(r.cpu().numpy(), wr)
    assert int(c) == wc and ids.tolist() == [int(x) for x in wids]
    return flags


@pytest.mark.parametrize("S,mb,bs,nb", [(1, 1, 16, 1), (3, 8, 64, 30), (40, 33, 16, 700), (64, 513, 64, 20000), (700, 300, 32, 70000)])
def test_free(S, mb, bs, nb):
    rng = np.random.default_rng(S + nb)
    table, refs, free, count, lens = _state(rng, S, mb, bs, nb)
    seqs = rng.permutation(S)[:max(1, 2 * S // 3)]
    assert _free(table, bs, nb, refs, seqs, free, count) == 0
    assert _free(table, bs, nb, refs, seqs, free, count, None, [int(rng.integers(0, n + 1)) for n in lens[seqs]]) == 0
    lo = [int(rng.integers(0, n + 1)) for n in lens[seqs]]
    hi = [int(rng.integers(0, n + 40)) for n in lens[seqs]]           # (some of them empty)
    assert _free(table, bs, nb, refs, seqs, free, count, lo, hi) == 0
    assert _free(table, bs, nb, refs, np.concatenate([seqs, seqs]), free, count) == 0   # named twice: once


def test_free_flags():
    rng = np.random.default_rng(9)
    S, mb, bs, nb = 6, 5, 16, 24
    table, refs, free, count, lens = _state(rng, S, mb, bs, nb)
    seqs = list(range(S))
    held = int((refs[np.unique(table[table >= 0])] >= 0).sum())
    assert held > 2
    assert _free(table, bs, nb, refs, seqs, free[:count + held].copy(), count) == 0
    assert _free(table, bs, nb, refs, seqs + [6, -1], free, count) == kvr.DEV_BAD_SEQ
    assert _free(table, bs, nb, refs, seqs, free, count, [0] * S, [2 ** 62] * S) == 0     # all kept
    assert _free(table, bs, nb, refs, seqs, free, count, [2 ** 62] * S, [-(2 ** 62)] * S) == 0
    wrong = table.copy()
    wrong[0, 3], wrong[1, 4] = nb, -9
    assert _free(wrong, bs, nb, refs, seqs, free, count) == kvr.DEV_BAD_BLOCK
    # no room: nothing is listed, and the next call with room lists it
    t, r, ids, c = _t(table), _t(refs), _t(free[:count + held - 1]), _t([count])
    kvr.kv_pages_free(t, nb, bs, r, _t(seqs), ids, c)
    assert kvr.device_status() == kvr.DEV_FREE_FULL and int(c) == count
    big = _t(free)
    kvr.kv_pages_free(t, nb, bs, r, _t([0]), big, c)
    assert kvr.device_status() == 0 and int(c) == nb and sorted(big.tolist()) == list(range(nb)) and not r.any()


# -- fork ----------------------------------------------------------------------------------------------------------------

def _fork(table, bs, nb, refs, src, dst, lens, free, count, in_place=True):
    n = len(src)
    t, r, ids, c = _t(table), _t(refs), _t(free), _t([count])
    a, b, k = torch.full((n,), 77, dtype=torch.int32, device=DEV), torch.full((n,), 77, dtype=torch.int32, device=DEV), _t([77])
    left = c if in_place else _t([-99])
    kvr.kv_pages_fork(t, nb, bs, r, _t(src), _t(dst), _t(lens, torch.int64), ids, c, a, b, k,
                      free_count_out=None if in_place else left)
    flags = kvr.device_status()
    wt, wr, pairs, wc, wf = ops.fork(table, bs, refs, src, dst, lens, free, count)
    assert flags == wf
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(r.cpu().numpy(), wr)
    assert int(left) == wc and int(k) == len(pairs) and ids.tolist() == [int(x) for x in free]
    if not in_place:
        assert int(c) == count
    assert list(zip(a.tolist(), b.tolist()))[:len(pairs)] == pairs
    assert a[len(pairs):].eq(77).all()
    return flags


@pytest.mark.parametrize("S,mb,bs,nb,n", [(2, 1, 16, 4, 1), (9, 8, 64, 80, 5), (150, 33, 16, 3000, 100), (64, 513, 64, 20000, 63),
                                          (9000, 6, 32, 60000, 8192)])
def test_fork(S, mb, bs, nb, n):
    rng = np.random.default_rng(S + n)
    table, refs, free, count, lens = _state(rng, S, mb, bs, nb, shared=0.0)
    live = np.nonzero(lens)[0]
    live = live[:max(1, min(len(live), S - n))]
    if len(live) == 0:
        live = np.array([0])
        count -= 1
        table[0, 0], lens[0] = free[count], bs
    dst = np.setdiff1d(np.arange(S), live)[:n]
    dst = rng.permutation(dst)
    src = rng.choice(live, len(dst))
    cut = [int(rng.integers(0, lens[s] + 1)) for s in src]
    cut = [c // bs * bs if rng.random() < 0.3 else c for c in cut]
    for in_place in (True, False):
        assert _fork(table, bs, nb, refs, src, dst, cut, free, count, in_place) == 0


def test_fork_flags():
    rng = np.random.default_rng(3)
    S, mb, bs, nb = 8, 4, 16, 40
    table, refs = np.full((S, mb), -1, np.int32), np.zeros(nb, np.int32)
    free = rng.permutation(nb).astype(np.int32)
    table[0, :3], table[1, :2] = free[37:40], free[35:37]
    count = 35
    call = lambda **kw: _fork(**{**dict(table=table, bs=bs, nb=nb, refs=refs, src=[0, 0, 1], dst=[2, 3, 4], lens=[40, 48, 17],
                                        free=free, count=count), **kw})
    assert call() == 0
    assert call(count=2) == 0 and call(count=1) == kvr.DEV_NO_BLOCKS and call(count=0) == kvr.DEV_NO_BLOCKS
    assert call(count=-1) == kvr.DEV_NO_BLOCKS and call(count=nb + 1) == kvr.DEV_NO_BLOCKS
    assert call(lens=[40, 32, 16], count=1) == 0                       # one part of a block alone
    assert call(src=[0, 8, -1]) == kvr.DEV_BAD_SEQ and call(dst=[2, 8, -1]) == kvr.DEV_BAD_SEQ
    assert call(dst=[2, 0, 4]) == kvr.DEV_BAD_SEQ                      # onto itself
    assert call(lens=[-1, 65, 2 ** 62]) == kvr.DEV_BAD_POS
    assert call(lens=[0, 64, 64]) == kvr.DEV_BAD_BLOCK                 # src does not hold all of it
    assert call(lens=[0, 0, 0], count=0) == 0
    bad = free.copy()
    bad[count - 1], bad[count - 2] = nb, -4
    assert call(free=bad) == kvr.DEV_BAD_BLOCK
    assert call(lens=[60, 50, 50]) == kvr.DEV_BAD_BLOCK                # the last block to be copied is not there
    assert call(src=[], dst=[], lens=[]) == 0


# -- compact -------------------------------------------------------------------------------------------------------------

def _compact(table, nb, refs, free, count, limit=0, in_place=True):
    t, r, ids, c = _t(table), _t(refs), _t(free), _t([count])
    a, b, k = (torch.full((max(nb // 2, 1),), 77, dtype=torch.int32, device=DEV) for _ in range(3))
    k = k[:1].contiguous()
    outs = (t, r, ids) if in_place else (torch.full_like(t, 55), torch.full_like(r, 55), torch.full_like(ids, 55))
    kw = {} if in_place else dict(table_out=outs[0], refs_out=outs[1], free_ids_out=outs[2])
    kvr.kv_pages_compact(t, nb, r, ids, c, a, b, k, limit=limit, **kw)
    flags = kvr.device_status()
    wt, wr, wids, pairs, wf = ops.compact(table, refs, free, count, limit)
    assert flags == wf and int(c) == count and int(k) == len(pairs)
    assert np.array_equal(outs[0].cpu().numpy(), wt) and np.array_equal(outs[1].cpu().numpy(), wr)
    if 0 <= count <= len(free):
        assert outs[2][:count].tolist() == wids
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert list(zip(a.tolist(), b.tolist()))[:len(pairs)] == pairs
    assert a[len(pairs):].eq(77).all() and b[len(pairs):].eq(77).all()
    return flags


@pytest.mark.parametrize("S,mb,nb", [(1, 1, 1), (1, 3, 2), (5, 8, 40), (40, 33, 1023), (70, 300, 8192), (100, 513, 30011)])
def test_compact(S, mb, nb):
    rng = np.random.default_rng(S + nb)
    bs = 16
    table, refs, free, count, lens = _state(rng, S, mb, bs, nb)
    used = nb - count
    for limit in (0, used, (used + nb) // 2, nb, nb + 100):
        for in_place in (True, False):
            assert _compact(table, nb, refs, free, count, limit, in_place) == 0
    if used > 1:
        assert _compact(table, nb, refs, free, count, used - 1, False) == kvr.DEV_NO_BLOCKS


def test_compact_edges():
    nb, S, mb = 20, 3, 6
    table, refs = np.full((S, mb), -1, np.int32), np.zeros(nb, np.int32)
    every = np.arange(nb, dtype=np.int32)
    assert _compact(table, nb, refs, every, nb) == 0                            # nothing used
    table.reshape(-1)[:] = np.arange(18)
    assert _compact(table, nb, refs, every, 0) == 0                             # nothing free (two blocks in no table)
    refs[3], refs[19] = 2, 5
    free = np.array([0, 7, 18] + [-1] * 17, np.int32)
    stale = table.copy()
    stale[2, 5], stale[2, 4] = nb + 3, -8                                       # kept as they are
    for in_place in (True, False):
        assert _compact(stale, nb, refs, free, 3, 0, in_place) == 0             # entries 0 and 7 name free blocks
        for bad, c in ((np.array([0, 7, 7], np.int32), 3), (np.array([0, 20, 7], np.int32), 3), (np.array([-1, 2, 7], np.int32), 3),
                       (free, 21), (free, -1), (free[:2].copy(), 3)):
            assert _compact(table, nb, refs, bad, c, 0, in_place) == kvr.DEV_BAD_BLOCK


def test_the_largest_pool():
    """2^20 blocks, the most that a compaction takes: the bit set at its full size."""
    rng = np.random.default_rng(8)
    nb, S, mb, bs = 1 << 20, 40, 60, 16
    free, used = rng.permutation(nb).astype(np.int32), 0
    table, refs = np.full((S, mb), -1, np.int32), np.zeros(nb, np.int32)
    count = nb - 500
    for s in range(20):
        m = int(rng.integers(1, 25))
        table[s, :m] = free[count + used:count + used + m]
        used += m
    refs[free[count:count + used]] = rng.integers(0, 3, used)
    for limit in (0, 500, nb // 2, nb - 1, nb):
        assert _compact(table, nb, refs, free, count, limit, False) == 0
    assert _compact(table, nb, refs, free, count, 499) == kvr.DEV_NO_BLOCKS
    assert _compact(table, nb, refs, free, count) == 0
    refs[:] = 0
    assert _free(table, bs, nb, refs, list(range(S)), free, count) == 0
    assert _fork(table, bs, nb, refs, [0, 1, 0], [30, 31, 32], [16, 5, 9], free, count) == 0
    nearly = np.arange(nb - 1, 0, -1, dtype=np.int32)                           # one block in use, the first; then the last
    table[:] = -1
    assert _compact(table, nb, refs, nearly, nb - 1) == 0
    table[3, 2] = nb - 1
    assert _compact(table, nb, refs, np.arange(nb, dtype=np.int32), nb - 1) == 0


def test_two_streams_at_once():
    """Two tables, each by a stream of its own, at the same time."""
    S, mb, bs, nb = 60, 40, 16, 3000
    runs = []
    for seed in (41, 42):
        rng = np.random.default_rng(seed)
        table, refs, free, count, lens = _state(rng, S, mb, bs, nb, shared=0.0)
        live = np.nonzero(lens)[0]
        dst = np.nonzero(lens == 0)[0][:20]
        src = rng.choice(live, len(dst))
        cut = [int(rng.integers(0, lens[s] + 1)) for s in src]
        runs.append(dict(t=_t(table), r=_t(refs), ids=_t(free), c=_t([count]), src=_t(src), dst=_t(dst), cut=_t(cut, torch.int64),
                         a=_t([0] * nb), b=_t([0] * nb), k=_t([0]), was=(table, refs, free, count, src, dst, cut)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, st in zip(runs, streams):
            kvr.kv_pages_free(x["t"], nb, bs, x["r"], x["dst"], x["ids"], x["c"], stream=st)
        for x, st in zip(runs, streams):
            kvr.kv_pages_fork(x["t"], nb, bs, x["r"], x["src"], x["dst"], x["cut"], x["ids"], x["c"], x["a"], x["b"], x["k"], stream=st)
        for x, st in zip(runs, streams):
            kvr.kv_pages_compact(x["t"], nb, x["r"], x["ids"], x["c"], x["a"], x["b"], x["k"], stream=st)
    torch.cuda.synchronize()
    assert kvr.device_status() == 0
    for x in runs:
        table, refs, free, count, src, dst, cut = x["was"]
        free = list(free)
        for _ in range(10):
            table, refs, free, count, f = ops.free(table, bs, refs, dst, free, count)
            table, refs, _, count, g = ops.fork(table, bs, refs, src, dst, cut, free, count)
            table, refs, left, pairs, h = ops.compact(table, refs, free, count)
            free[:count] = left
            assert f == g == h == 0
        assert np.array_equal(x["t"].cpu().numpy(), table) and np.array_equal(x["r"].cpu().numpy(), refs)
        assert int(x["c"]) == count and x["ids"][:count].tolist() == left and int(x["k"]) == len(pairs)


# -- copy ----------------------------------------------------------------------------------------------------------------

def _pools(gen, nb, hkv, bs, kinds):
    bt = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    out = []
    for kind in kinds:
        if kind == 16:
            out.append(kvr.PagedLayout(*(torch.randn(nb, hkv, bs, d, generator=gen, device=DEV).bfloat16() for d in (192, 128)), bt))
        else:
            cls = kvr.Kv4Layout if kind == 4 else kvr.Kv8Layout
            out.append(cls(torch.randint(0, 256, (nb, hkv, bs // 16, cls.TILE), generator=gen, device=DEV, dtype=torch.uint8), bt))
    return out


@pytest.mark.parametrize("nb,hkv,bs,kinds,n", [(3, 1, 16, [8], 1), (50, 2, 48, [16, 4, 8], 20), (9, 8, 1024, [16], 4),
                                               (400, 1, 16, [8] * 130, 100), (300, 4, 64, [8, 16], 150)])
def test_copy(nb, hkv, bs, kinds, n):
    gen = torch.Generator(device=DEV).manual_seed(nb)
    pools = _pools(gen, nb, hkv, bs, kinds)
    order = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    src, dst = order[:n].clone(), order[nb - n:].clone()
    src[-1] = src[0]                                                            # two copies of one block
    for count, flags in ((n, 0), (n // 2, 0), (0, 0), (-5, 0), (n + 1000, 0)):
        want = [[x.clone() for x in p.tensors()[:-1]] for p in pools]
        m = max(min(count, n), 0)
        for w in want:
            for x in w:
                x[dst[:m].long()] = x[src[:m].long()]
        kvr.kv_pages_copy(pools, src, dst, _t([count]))
        assert kvr.device_status() == flags
        for p, w in zip(pools, want):
            for x, y in zip(p.tensors(), w):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), count


def test_copy_skips_what_is_no_block():
    gen = torch.Generator(device=DEV).manual_seed(5)
    pools = _pools(gen, 6, 2, 32, [16, 8])
    want = [[x.clone() for x in p.tensors()[:-1]] for p in pools]
    for w in want:
        for x in w:
            x[3] = x[1]
    kvr.kv_pages_copy(pools, _t([-1, 6, 1, 0, 2 ** 31 - 1]), _t([2, 4, 3, 6, 5]), _t([5]))
    assert kvr.device_status() == kvr.DEV_BAD_BLOCK
    for p, w in zip(pools, want):
        for x, y in zip(p.tensors(), w):
            assert torch.equal(x, y)


def test_copy_past_4_gb():
    hkv, bs = 8, 1024                                                            # 2000 blocks of 3 MB of K and 2 MB of V
    k = torch.empty(2000, hkv, bs, 192, dtype=torch.bfloat16, device=DEV)
    v = torch.empty(2000, hkv, bs, 128, dtype=torch.bfloat16, device=DEV)
    pool = kvr.PagedLayout(k, v, torch.zeros(1, 1, dtype=torch.int32, device=DEV))
    k[1999], v[1999] = 3.0, 5.0
    k[7], v[7] = 2.0, 4.0
    k[1998] = v[1998] = k[0] = v[0] = 0.0
    kvr.kv_pages_copy(pool, _t([1999, 7]), _t([0, 1998]), _t([2]))
    assert k[0].eq(3).all() and v[0].eq(5).all() and k[1998].eq(2).all() and v[1998].eq(4).all()
    assert kvr.device_status() == 0


# -- together ------------------------------------------------------------------------------------------------------------


def test_a_run_of_them_together():
    """A prompt is written, forked into samples that go on by themselves (each decode step: grow, append, decode, in one
    captured graph), two of them end, one is forked again from the middle, the pool is shrunk; at every point each
    sample's decode over the shared pool is what the same tokens give in a pool of their own, and the bf16 pool that
    goes along under the same table holds the same rows as one written straight."""
    gen = torch.Generator(device=DEV).manual_seed(17)
    hkv, G, bs, S, mb, nb = 2, 8, 32, 6, 12, 60
    table = kvr.rope_table(1e7, mb * bs)
    bt = torch.full((S, mb), -1, dtype=torch.int32, device=DEV)
    p8 = kvr.Kv8Layout(torch.full((nb, hkv, bs // 16, kvr.KV8_TILE), 0xFF, dtype=torch.uint8, device=DEV), bt)
    p16 = kvr.PagedLayout(torch.full((nb, hkv, bs, 192), float("nan"), dtype=torch.bfloat16, device=DEV),
                          torch.full((nb, hkv, bs, 128), float("nan"), dtype=torch.bfloat16, device=DEV), bt)
    free, count = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32), _t([nb])
    refs = torch.zeros(nb, dtype=torch.int32, device=DEV)
    ca, cb, cc = (torch.zeros(nb, dtype=torch.int32, device=DEV) for _ in range(3))
    cc = cc[:1].contiguous()
    K = {s: torch.zeros(0, hkv, 192, dtype=torch.bfloat16, device=DEV) for s in range(S)}   # each sequence's own rows
    V = {s: torch.zeros(0, hkv, 128, dtype=torch.bfloat16, device=DEV) for s in range(S)}
    cuts = {s: [] for s in range(S)}                                                       # and the chunks they came in

    def rows(T):
        return (torch.randn(T, hkv, 192, generator=gen, device=DEV).bfloat16(), torch.randn(T, hkv, 128, generator=gen, device=DEV).bfloat16())

    def write(seqs, n, k, v, lens):
        T = sum(n)
        cu, pos = torch.empty(len(n) + 1, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)
        rs, sl = torch.empty(T, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)
        kvr.kv_pages_grow(bt, nb, bs, seqs, lens, _t(n), free, count, cu, pos, rs, sl)
        kvr.kv8_append_rope(k, v, cu, lens, seqs, table, VS, p8)
        kvr.kv_ring_append_rope(k, v, pos, rs, table, VS, p16)

    def note(seqs, n, k, v):
        at = 0
        for s, c in zip(seqs, n):
            K[s], V[s] = torch.cat([K[s], k[at:at + c]]), torch.cat([V[s], v[at:at + c]])
            cuts[s].append(c)
            at += c

    def check(live):
        q = torch.randn(len(live), hkv * G, 192, generator=gen, device=DEV).bfloat16()
        pos = _t([K[s].shape[0] - 1 for s in live], torch.int64)
        got8 = kvr.full_attn_decode_kv8(q, pos, _t(live), p8, table, SCALE, mb * bs)
        got16 = kvr.full_attn_decode(q, pos, _t(live), p16, table, SCALE, mb * bs)
        own8 = kvr.Kv8Layout.contiguous(len(live), hkv, mb * bs, block_size=bs)
        own16 = kvr.PagedLayout.contiguous(len(live), hkv, mb * bs, block_size=bs)
        for i, s in enumerate(live):
            at = 0
            for c in cuts[s]:
                kvr.kv8_append_rope(K[s][at:at + c].contiguous(), V[s][at:at + c].contiguous(), _t([0, c]), _t([at], torch.int64), _t([i]),
                                    table, VS, own8)
                at += c
            kvr.kv_ring_append_rope(K[s], V[s], torch.arange(at, device=DEV), torch.full((at,), i, dtype=torch.int32, device=DEV),
                                    table, VS, own16)
        mine = torch.arange(len(live), dtype=torch.int32, device=DEV)
        assert torch.equal(got8, kvr.full_attn_decode_kv8(q, pos, mine, own8, table, SCALE, mb * bs))
        assert torch.equal(got16, kvr.full_attn_decode(q, pos, mine, own16, table, SCALE, mb * bs))
        # the 8-bit values are within half a step (a 250th of the largest, |v| < 4) and twice that where a scale grew: a
        # score moves by 192 products of such steps at random, the values by a step: 0.1 covers both many times over
        assert float((got8.float() - got16.float()).abs().max()) <= 0.1
        assert kvr.device_status() == 0
        held = torch.bincount(bt[bt >= 0].long(), minlength=nb)
        gone = torch.zeros(nb, dtype=torch.int64, device=DEV)
        gone[free[:int(count)].long()] = 1
        assert torch.equal(held + gone, torch.where(gone > 0, 1, refs.long() + 1))

    k, v = rows(75)
    write(_t([1]), [75], k, v, _t([0], torch.int64))
    note([1], [75], k, v)
    check([1])
    # three samples of the first 75 positions, one of the first 64 (two whole blocks)
    src, dst, n = [1, 1, 1], [0, 4, 5], [75, 75, 64]
    kvr.kv_pages_fork(bt, nb, bs, refs, _t(src), _t(dst), _t(n, torch.int64), free, count, ca, cb, cc)
    kvr.kv_pages_copy([p8, p16], ca, cb, cc)
    for s, d, m in zip(src, dst, n):
        K[d], V[d], cuts[d] = K[s][:m], V[s][:m], [m]
    assert int(cc) == 2 and int(count) == nb - 5 and int(refs.sum()) == 6
    check([0, 1, 4, 5])
    # each goes on by itself, in a captured graph
    live = [0, 1, 4, 5]
    seqs, lens = _t(live), torch.zeros(4, dtype=torch.int64, device=DEV)
    sk, sv = rows(4)
    cu, pos = torch.empty(5, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int64, device=DEV)
    rs, sl, one = torch.empty(4, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int64, device=DEV), _t([1] * 4)

    def step():
        kvr.kv_pages_grow(bt, nb, bs, seqs, lens, one, free, count, cu, pos, rs, sl)
        kvr.kv8_append_rope(sk, sv, cu, lens, seqs, table, VS, p8)
        kvr.kv_ring_append_rope(sk, sv, pos, rs, table, VS, p16)

    lens.copy_(_t([K[s].shape[0] for s in live], torch.int64))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(30):
        a, b = rows(4)
        sk.copy_(a)
        sv.copy_(b)
        lens.copy_(_t([K[s].shape[0] for s in live], torch.int64))
        g.replay()
        note(live, [1] * 4, a, b)
    check(live)
    # two of them end, and the prompt itself is cut to 40 positions; what others hold stays
    kvr.kv_pages_free(bt, nb, bs, refs, _t([0, 5]), free, count)
    kvr.kv_pages_free(bt, nb, bs, refs, _t([1]), free, count, keep_hi=_t([40], torch.int64))
    K[1], V[1], cuts[1] = K[1][:40], V[1][:40], None
    # (the cut's tile keeps the scale that later rows gave it, so the prompt is compared by its bf16 rows alone)
    check([4])
    # a sample of a sample, from inside its last tiles
    kvr.kv_pages_fork(bt, nb, bs, refs, _t([4]), _t([2]), _t([96], torch.int64), free, count, ca, cb, cc)
    kvr.kv_pages_copy([p8, p16], ca, cb, cc)
    assert int(cc) == 0
    K[2], V[2] = K[4][:96], V[4][:96]
    at, cuts[2] = 0, []
    for c in cuts[4]:
        if at < 96:
            cuts[2].append(min(c, 96 - at))
            at += c
    check([2, 4])
    # the pool shrinks to what is used
    used = nb - int(count)
    kvr.kv_pages_compact(bt, nb, refs, free, count, ca, cb, cc)
    kvr.kv_pages_copy([p8, p16], ca, cb, cc)
    assert int(bt.max()) < used and int(free[:nb - used].min()) == used
    check([2, 4])
    small = [kvr.Kv8Layout(p8.data[:used].clone(), bt), kvr.PagedLayout(p16.k[:used].clone(), p16.v[:used].clone(), bt)]
    q = torch.randn(2, hkv * G, 192, generator=gen, device=DEV).bfloat16()
    args = (q, _t([95, K[4].shape[0] - 1], torch.int64), _t([2, 4]))
    assert torch.equal(kvr.full_attn_decode_kv8(*args, small[0], table, SCALE, mb * bs), kvr.full_attn_decode_kv8(*args, p8, table, SCALE, mb * bs))
    assert torch.equal(kvr.full_attn_decode(*args, small[1], table, SCALE, mb * bs), kvr.full_attn_decode(*args, p16, table, SCALE, mb * bs))
    # and a new request is served from the free list's lowest blocks
    k, v = rows(33)
    write(_t([3]), [33], k, v, _t([0], torch.int64))
    note([3], [33], k, v)
    assert sorted(bt[3][:2].tolist()) == [used, used + 1]
    check([2, 3, 4])


def test_captured_beam_step_replays():
    """Free, fork and copy in one graph, replayed with other parents and lengths."""
    rng = np.random.default_rng(21)
    S, mb, bs, nb = 10, 6, 16, 64
    gen = torch.Generator(device=DEV).manual_seed(3)
    table, refs = np.full((S, mb), -1, np.int32), np.zeros(nb, np.int32)
    free, count = np.arange(nb, dtype=np.int32), nb
    for s in (0, 1):
        for j in range(mb):
            count -= 1
            table[s, j] = free[count]
    pools = _pools(gen, nb, 1, bs, [8, 4])
    t, r, ids, c = _t(table), _t(refs), _t(free), _t([count])
    src, dst, lens = _t([0] * 4), _t([2, 3, 4, 5]), _t([20] * 4, torch.int64)
    a, b, k = _t([0] * 4), _t([0] * 4), _t([0])

    def beam():
        kvr.kv_pages_free(t, nb, bs, r, dst, ids, c)
        kvr.kv_pages_fork(t, nb, bs, r, src, dst, lens, ids, c, a, b, k)
        kvr.kv_pages_copy(pools, a, b, k)

    beam()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        beam()
    torch.cuda.synchronize()
    # the state as the first, eager step left it
    tab, ref, free, count = t.cpu().numpy(), r.cpu().numpy(), ids.tolist(), int(c)
    for _ in range(20):
        ws, wl = rng.integers(0, 2, 4), rng.integers(0, mb * bs + 1, 4)
        src.copy_(_t(ws))
        lens.copy_(_t(wl, torch.int64))
        old = [p.data.clone() for p in pools]
        g.replay()
        torch.cuda.synchronize()
        tab, ref, free, count, f = ops.free(tab, bs, ref, [2, 3, 4, 5], free, count)
        assert f == 0
        tab, ref, pairs, count, f = ops.fork(tab, bs, ref, ws, [2, 3, 4, 5], wl, free, count)
        assert f == 0 and kvr.device_status() == 0
        assert np.array_equal(t.cpu().numpy(), tab) and np.array_equal(r.cpu().numpy(), ref) and int(c) == count
        assert ids.tolist()[:count] == free[:count] and int(k) == len(pairs)
        for p, o in zip(pools, old):
            for x, y in pairs:
                o[y] = o[x]
            assert torch.equal(p.data, o)


def test_on_another_stream():
    rng = np.random.default_rng(30)
    S, mb, bs, nb = 20, 30, 16, 500
    table, refs, free, count, lens = _state(rng, S, mb, bs, nb)
    t, r, ids, c = _t(table), _t(refs), _t(free), _t([count])
    a, b, k = _t([0] * nb), _t([0] * nb), _t([0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kvr.kv_pages_free(t, nb, bs, r, _t(range(10)), ids, c, stream=st)
    kvr.kv_pages_compact(t, nb, r, ids, c, a, b, k, stream=st)
    st.synchronize()
    wt, wr, wf, wc, _ = ops.free(table, bs, refs, range(10), free, count)
    wt, wr, wl, pairs, _ = ops.compact(wt, wr, wf, wc)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(r.cpu().numpy(), wr) and ids[:wc].tolist() == wl
    assert int(k) == len(pairs) and kvr.device_status() == 0
