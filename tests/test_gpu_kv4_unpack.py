"""kv4_unpack where T is far above the rows of a call (the default for a block table wider than its pool), and calls
whose units go round: every bit against the fp64 values of the codes."""
import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import kv4 as o4

pytestmark = pytest.mark.gpu
DEV = "cuda"


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


def _ints(v, t):
    return torch.tensor(v, dtype=t, device=DEV)


def _filled(gen, S, hkv, n, bs, table):
    pool = kvr.Kv4Layout.contiguous(S, hkv, n, block_size=bs)
    for s in range(S):
        k = torch.randn(n, hkv, 192, generator=gen, device=DEV).bfloat16()
        v = torch.randn(n, hkv, 128, generator=gen, device=DEV).bfloat16()
        kvr.kv4_append_rope(k, v, torch.arange(n, device=DEV), torch.full((n,), s, dtype=torch.int32, device=DEV), table,
                            0.707, pool)
    return pool


def _want(pool, s, lo, n):
    """Rows [n, hkv, 192], [n, hkv, 128]: fp64 -> fp32 -> bf16, as the kernel's sum and store."""
    pl = [o4.places(r) for r in range(16)]
    at = [torch.tensor(np.array([p[i] for p in pl]), device=DEV) for i in range(6)]
    hi = (torch.arange(192, device=DEV) % 2 * 4).to(torch.uint8)
    tiles = pool.data[pool.block_table[s].long()].transpose(1, 2).flatten(0, 1)[lo // 16:-(-(lo + n) // 16)]
    out = []
    for codes, scales, minima, w in ((0, 2, 5, 192), (1, 3, 4, 128)):
        half = lambda a: torch.stack([tiles[..., a], tiles[..., a + 1]], -1).contiguous().view(torch.float16)[..., 0].double()
        u = ((tiles[..., at[codes]] >> hi[:w]) & 15).double()
        x = half(at[minima]).repeat_interleave(64, -1) + half(at[scales]).repeat_interleave(64, -1) * u
        out.append(x.float().bfloat16().transpose(1, 2).flatten(0, 1)[lo % 16:lo % 16 + n])
    return out


def _rows(pages, s, n):
    k = pages.k[pages.block_table[s].long()[:-(-n // pages.block_size)]].transpose(1, 2).flatten(0, 1)[:n]
    v = pages.v[pages.block_table[s].long()[:-(-n // pages.block_size)]].transpose(1, 2).flatten(0, 1)[:n]
    return k, v


@pytest.mark.parametrize("hkv,S,mb", [(16, 64, 1 << 15), (3, 9, 40), (5, 2000, 300)])
def test_default_rows_of_a_wide_table(table, hkv, S, mb):
    """Tables that span 2^31 positions (of 16 heads: more units than 31 bits count), thousands and millions of them, over
    a pool of six blocks."""
    gen = torch.Generator(device=DEV).manual_seed(hkv)
    src = _filled(gen, 2, hkv, 1500, 64, table)
    bs = 1024
    bt = torch.full((S, mb), -1, dtype=torch.int32, device=DEV)
    bt[S - 1, :2], bt[1, :2] = _ints([4, 2], torch.int32), _ints([0, 3], torch.int32)
    pages = kvr.PagedLayout(torch.full((6, hkv, bs, 192), 9.0, dtype=torch.bfloat16, device=DEV),
                            torch.full((6, hkv, bs, 128), 9.0, dtype=torch.bfloat16, device=DEV), bt)
    call = lambda lo, cu, dst: kvr.kv4_unpack(src, _ints([1, 0, 0], torch.int32), _ints(lo, torch.int64),
                                              _ints(cu, torch.int32), pages, dst_seqs=_ints(dst, torch.int32))
    call([0, 7, 0], [0, 1500, 2493, 2493], [S - 1, 1, 0])
    assert kvr.device_status() == 0
    for a, b in zip(_rows(pages, S - 1, 1500), _want(src, 1, 0, 1500)):
        assert torch.equal(a, b)
    for a, b in zip(_rows(pages, 1, 1000), _want(src, 0, 7, 993)):
        assert torch.equal(a[7:], b) and (a[:7] == 9).all()
    assert (pages.k[1] == 9).all() and (pages.k[5] == 9).all()
    # what is flagged of a call that goes round is what is flagged of a small one
    before = pages.k.clone()
    call([0, -1, 0], [0, 100, 90, 200], [S - 1, 1, 1])
    assert kvr.device_status() & kvr.DEV_BAD_ROWS
    call([-5, 0, 1 << 60], [0, 100, 100, 200], [S - 1, 1, 1])
    assert kvr.device_status() == kvr.DEV_BAD_POS
    call([0, 0, 0], [0, 0, 0, 16], [S - 1, 1, S])
    assert kvr.device_status() == kvr.DEV_BAD_SEQ
    call([0, 0, 0], [0, 0, 0, 0], [S - 1, 1, 0])
    assert kvr.device_status() == 0
    assert torch.equal(pages.k[[1, 2, 3, 5]], before[[1, 2, 3, 5]])


def test_units_that_go_round(table):
    """More units than a call takes at once, in chunks that start and end inside tiles."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    hkv, n = 8, 100001
    src = _filled(gen, 1, hkv, n, 48, table)
    lo = [3, 0, 17, 99999, 5000]
    rows = [99990, 0, 60001, 2, 95000]
    reps = 6                                        # 1.5 million rows: 771,000 units of 524,288 warps
    cu = np.concatenate([[0], np.cumsum(rows * reps)]).tolist()
    m = len(rows) * reps
    dst = kvr.LinearLayout.empty(cu[-1] + 5, hkv)
    dst.k[cu[-1]:], dst.v[cu[-1]:] = 9, 9
    kvr.kv4_unpack(src, torch.zeros(m, dtype=torch.int32, device=DEV), _ints(lo * reps, torch.int64), _ints(cu, torch.int32), dst)
    assert kvr.device_status() == 0
    for e in range(len(rows)):
        k, v = _want(src, 0, lo[e], rows[e])
        for i in range(e, m, len(rows)):
            assert torch.equal(dst.k[cu[i]:cu[i + 1]], k) and torch.equal(dst.v[cu[i]:cu[i + 1]], v), i
    assert (dst.k[cu[-1]:] == 9).all() and (dst.v[cu[-1]:] == 9).all()
