"""Batches of chunks of the 8-bit pool whose cu_rows is out of order, or runs past the
rows that there are: the call says so, whatever form its units take, and up to 64 chunks
those ahead of the place are written as if there were no others."""
import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import kv8 as o8

from test_gpu_kv8 import DEV, VS, _append, _built, _gen, _ints, _kv, _oracle_append, _pool, table  # noqa: F401

pytestmark = pytest.mark.gpu


def _served(cu, T):
    """How many chunks lie ahead of the first that is out of order."""
    ok = [0 <= a <= b <= T for a, b in zip(cu, cu[1:])]
    return ok.index(False) if False in ok else len(ok)


def _filled(gen, n, first, hkv, cap, table):
    pool = _pool(gen, n, hkv, cap, 16, fill=0x21)
    T = int(sum(first))
    k, v = _kv(gen, max(T, 1), hkv)
    _append(pool, k, v, list(range(n)), [0] * n, list(first), table)
    return pool


def _check_append(pool, cu, T, first, hkv, gen, table, flags, served, seqs=None, lo=None, good=None):
    """The first `good` chunks (all) are the oracle's, those of `served`, or as they were; the others are not looked at."""
    n = len(cu) - 1
    seqs = list(range(n)) if seqs is None else seqs
    lo = list(first) if lo is None else lo
    want, bt = pool.data.cpu().numpy(), pool.block_table.cpu().numpy()
    k, v = _kv(gen, T, hkv)
    kvr.kv8_append_rope(k, v, _ints(cu, torch.int32), _ints(lo, torch.int64), _ints(seqs, torch.int32), table, VS, pool)
    said = kvr.device_status()
    assert said == flags if good in (None, n) else said & flags
    written = {}
    for i in served:
        _oracle_append(want, bt, k[cu[i]:cu[i + 1]], v[cu[i]:cu[i + 1]], [seqs[i]], [int(lo[i])], [cu[i + 1] - cu[i]], table,
                       written=written)
    got = pool.data.cpu().numpy()
    for blk in bt[n if good is None else good:].flatten():
        if 0 <= blk < len(got):
            got[blk] = want[blk] = 0
    assert o8.same(got, want, written)


def _check_unpack(pool, cu, T, hkv, flags, served, first=0):
    n = len(cu) - 1
    lo, seqs = [first] * n, list(range(n))
    out = kvr.LinearLayout(torch.full((T, hkv, 192), 7.0, dtype=torch.bfloat16, device=DEV),
                           torch.full((T, hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV))
    kvr.kv8_unpack(pool, _ints(seqs, torch.int32), _ints(lo, torch.int64), _ints(cu, torch.int32), out)
    said = kvr.device_status()
    assert said & flags if served < n else said == flags
    data, bt = pool.data.cpu().numpy(), pool.block_table.cpu().numpy()
    behind = np.zeros(T, bool)  # rows that a chunk behind the place names: its own, or the one's ahead
    for a, b in zip(cu[served:], cu[served + 1:]):
        behind[max(a, 0):max(b, 0)] = True
    for i in range(served):
        if cu[i] < cu[i + 1]:
            for h in range(hkv):
                keep = torch.from_numpy(~behind[cu[i]:cu[i + 1]])
                K, V, _ = o8.sequence(data, bt[i], h, first + cu[i + 1] - cu[i])
                for got, want in ((out.k, K), (out.v, V)):
                    assert torch.equal(got[cu[i]:cu[i + 1], h].cpu()[keep], torch.from_numpy(want[first:]).bfloat16()[keep]), i
    if served == n:
        assert (out.k[max(cu[-1], 0):] == 7).all() and (out.v[max(cu[-1], 0):] == 7).all()


ORDERS = {
    "past the rows": ([*range(13)], 9),
    "past the rows, by far": ([0, 1, 2, 3, 4, 5, 6, 7, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], 9),
    "a step back": ([0, 1, 2, 3, 4, 3, 4, 5, 6, 7, 8, 9, 10], 10),
    "back to the first": ([0, 1, 0, 1], 1),
    "negative first": ([-2, 0, 1], 1),
    "negative first of many": ([-1, *range(1, 12)], 12),
    "negative last": ([0, 1, 2, 3, 4, 5, 6, 7, 8, -4], 9),
    "back by more than a tile's units": ([0, 100, 0, 100], 100),
    "back behind a long one": ([0, 3, 90, 91, 20, 95, 100], 100),
    "empty ahead of the place": ([0, 0, 0, 1, 1, 0, 1], 1),
}


@pytest.mark.parametrize("name", list(ORDERS))
def test_out_of_order(table, name):
    cu, T = ORDERS[name]
    n, hkv, gen = len(cu) - 1, 2, _gen(len(name))
    first = [3 * i % 17 for i in range(n)]
    good = _served(cu, T)
    assert good < n
    most = max([1] + [cu[i + 1] - cu[i] for i in range(good)])
    pool = _filled(gen, n, first, hkv, 32 + most, table)
    _check_append(pool, cu, T, first, hkv, gen, table, kvr.DEV_BAD_ROWS, range(good), good=good)
    whole = _filled(gen, n, [most + 16] * n, hkv, 32 + most, table)
    _check_unpack(whole, cu, T, hkv, kvr.DEV_BAD_ROWS, good, first=5)


@pytest.mark.parametrize("hkv", [1, 5])
@pytest.mark.parametrize("n", [3, 33, 40, 64])
@pytest.mark.parametrize("mean", [1, 12])
def test_one_place_out_of_order(table, mean, n, hkv):
    """Batches in order but for one entry, anywhere, or for none: by row and by tile, one head a CTA and several."""
    rng, gen = np.random.default_rng(n + mean + hkv), _gen(n + mean + hkv)
    for case in range(4):
        rows = rng.integers(0, 2 * mean + 1, n)
        cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
        T = max(int(cu[-1]), 1)
        at = int(rng.integers(0, n + 1))
        if case == 0:
            cu[at] = -1 - int(rng.integers(0, 1000))
        elif case == 1:
            cu[at] = T + 1 + int(rng.integers(0, 1000))
        elif case == 2:
            cu[at] = int(rng.integers(0, T + 1))
        cu = cu.tolist()
        good = _served(cu, T)
        flags = kvr.DEV_BAD_ROWS if good < n else 0
        first = rng.integers(0, 20, n).tolist()
        # (chunk `at` may have got longer, up to all rows, and be in order)
        most = max([1] + [cu[i + 1] - cu[i] for i in range(good)])
        pool = _filled(gen, n, first, hkv, 20 + most, table)
        _check_append(pool, cu, T, first, hkv, gen, table, flags, range(good), good=good)
        whole = _filled(gen, n, [most + 3] * n, hkv, 20 + most, table)
        _check_unpack(whole, cu, T, hkv, flags, good, first=3)


@pytest.mark.parametrize("n", [65, 500, 5000, 20000])
def test_out_of_order_among_many(table, n):
    """Told of any batch, wherever the place is; past 64 chunks, which of the others are written is not said."""
    gen = _gen(n)
    for at, to in ((n // 2, 7), (n, n + 1), (n - 1, -1), (0, -1), (1, n + 5)):
        for each in (1, 20):
            T = n * each
            pool = _pool(gen, n, 1, 32, 16, fill=0x21)
            k, v = _kv(gen, T, 1)
            cu = torch.arange(n + 1, dtype=torch.int32, device=DEV) * each
            cu[at] = to if to < n else to + T - n
            P0, seqs = torch.zeros(n, dtype=torch.int64, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV)
            kvr.kv8_append_rope(k, v, cu, P0, seqs, table, VS, pool)
            assert kvr.device_status() & kvr.DEV_BAD_ROWS
            kvr.kv8_unpack(pool, seqs, P0, cu, kvr.LinearLayout.empty(T, 1))
            assert kvr.device_status() & kvr.DEV_BAD_ROWS


@pytest.mark.parametrize("n", [8, 70])
def test_single_rows_and_what_cannot_be_written(table, n):
    """A decode step's chunks of one row: padding, ids, positions and blocks that are not there, beside good ones."""
    gen, hkv = _gen(n), 2
    first = [(5 * i) % 31 for i in range(n)]
    pool = _filled(gen, n, first, hkv, 32, table)
    pool.block_table[6, first[6] // 16] = pool.num_blocks
    pool.block_table[2, first[2] // 16] = -1
    cu = list(range(n + 1))
    odd = {1: (n, None), 3: (None, 32), 4: (None, -1), 5: (-1, 1 << 60), 7: (-9, 0)}
    seqs = [odd[i][0] if i in odd and odd[i][0] is not None else i for i in range(n)]
    lo = [odd[i][1] if i in odd and odd[i][1] is not None else first[i] for i in range(n)]
    served = [i for i in range(n) if i not in odd and i not in (2, 6)]
    _check_append(pool, cu, n, first, hkv, gen, table, kvr.DEV_BAD_SEQ | kvr.DEV_BAD_POS | kvr.DEV_BAD_BLOCK, served, seqs, lo)
    # and with the one in the middle past the rows that there are
    cu[2 if n <= 64 else 70] = n + 1
    _check_append(pool, cu, n, first, hkv, gen, table, kvr.DEV_BAD_ROWS, [0] if n <= 64 else [], seqs, lo, good=1 if n <= 64 else 0)


@pytest.mark.parametrize("n,at", [(3, 1), (40, 30), (64, 20), (64, 63)])
@pytest.mark.parametrize("T", [1 << 12, 1 << 19, (1 << 21) + 5])
def test_out_of_order_with_far_more_rows_allowed(table, T, n, at):
    """T far above the rows, and the entries behind the place all below those ahead of it: a unit ahead of it is not taken for
    one behind all rows.  (At once, at once with most CTAs behind the rows, and in rounds; both quantised pools.)"""
    gen, hkv, each = _gen(n + at), 4, 50
    cu = [each * i for i in range(at + 1)] + [3 + i % 2 for i in range(n - at)]
    good = _served(cu, T)
    assert good == at
    seqs = torch.arange(n, dtype=torch.int32, device=DEV)
    lo = torch.zeros(n, dtype=torch.int64, device=DEV)
    k, v = _kv(gen, each * n, hkv)
    whole = torch.arange(n + 1, dtype=torch.int32, device=DEV) * each
    p8, p4 = (cls.contiguous(n, hkv, 64, block_size=64) for cls in (kvr.Kv8Layout, kvr.Kv4Layout))
    kvr.kv8_append_rope(k, v, whole, lo, seqs, table, VS, p8)
    kvr.kv4_append_rope(k, v, torch.arange(each, device=DEV).repeat(n), seqs.repeat_interleave(each), table, VS, p4)
    for pool, call in ((p8, kvr.kv8_unpack), (p4, kvr.kv4_unpack)):
        pages = [kvr.PagedLayout.contiguous(n, hkv, 64, block_size=64) for _ in range(2)]
        for p in pages:
            p.k.fill_(7)
            p.v.fill_(7)
        call(pool, seqs, lo, whole, pages[0], dst_seqs=seqs, T=max(T, each * n))
        assert kvr.device_status() == 0
        call(pool, seqs, lo, _ints(cu, torch.int32), pages[1], dst_seqs=seqs, T=T)
        assert kvr.device_status() & kvr.DEV_BAD_ROWS
        for a, b in zip(pages[0].tensors()[:2], pages[1].tensors()[:2]):
            assert torch.equal(a[:good], b[:good])
        assert (pages[0].k[:, :, each:] == 7).all() and not (pages[0].k[:, :, :each] == 7).all(-1).any()
