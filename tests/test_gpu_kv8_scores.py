"""The 8-bit decode under scores of every size, against fp64 attention over the
query as the kernel holds it: scaled, brought by a power of two to [2^14, 2^15)
and rounded once to fp16, which numpy does alike.  (The RoPE table is the identity
here: a product and a sum of the rotation may or may not be one instruction, and an
fp16 rounding could fall the other way.)  So no rounding of the query is in a
tolerance, which in scores of hundreds would let anything pass."""
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
LN2 = math.log(2.0)


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
    t = torch.zeros(1 << 14, 32, 2, device=DEV)
    t[..., 0] = 1.0
    return t


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(v, t):
    return torch.tensor(v, dtype=t, device=DEV)


def _pool(gen, k, v, table, bs=64):
    """One sequence of keys k [n, 1, 192] and values v [n, 1, 128], in pages of any order."""
    n = k.shape[0]
    mb = -(-n // bs)
    ids = torch.randperm(mb + 2, generator=gen, device=DEV)[:mb].to(torch.int32).reshape(1, mb)
    data = torch.full((mb + 2, 1, bs // 16, kvr.KV8_TILE), 0xFF, dtype=torch.uint8, device=DEV)
    pool = kvr.Kv8Layout(data, ids.contiguous())
    kvr.kv8_append_rope(k.contiguous(), v.contiguous(), _ints([0, n], torch.int32), _ints([0], torch.int64),
                        _ints([0], torch.int32), table, 1.0, pool)
    return pool


def _held(q):
    """q [..., 192] as the kernel holds it: its scores are in units of log 2."""
    y = (q.float().cpu().numpy() * (np.float32(SCALE) * np.float32(1.4426950408889634))).astype(np.float32)
    m = np.abs(y).max(-1, keepdims=True).astype(np.float64)
    e = np.where(m > 0, 14 - np.floor(np.log2(np.where(m > 0, m, 1.0))), 0.0)
    e = np.minimum(e, 126)
    return (y.astype(np.float64) * 2.0 ** e).astype(np.float16).astype(np.float64) / 2.0 ** e


def _decode(q, pos, pool, table, most):
    out = kvr.full_attn_decode_kv8(q, _ints(pos, torch.int64), _ints([0] * len(pos), torch.int32), pool, table, SCALE, most)
    assert kvr.device_status() == 0
    return out.double().cpu().numpy()


def _values(pool, n):
    return o8.sequence(pool.data.cpu().numpy(), pool.block_table[0].cpu().numpy(), 0, n)


def _check(got, q, pos, pool, n, what=""):
    """Every row against fp64.  The output is rounded by half a bf16 step, 2^-8 |o|.  A score is twelve sums each cut off
    below 2^-23 of sum |q||k| at most, two roundings of 2^-24 and a reference's as much: less than 2^-19 sum |q||k|, by which
    a weight and the sum of weights each move as exponentials.  A weight is rounded to fp16 (2^-11 of it), the sums over keys
    are cut off below 2^-23 once a tile: under 2^-10 sum p |v| and 2^-20 |v|_max."""
    K, V, ok = _values(pool, n)
    held, cs = _held(q), np.stack([np.ones(32), np.zeros(32)], 1)
    vmax = np.abs(V).max()
    for b, p in enumerate(pos):
        want, a, w = attend(held[b], p, K, V, ok, cs, LN2)
        err = np.abs(got[b] - want)
        move = np.exp(2 * 2.0 ** -19 * a[:, None]) - 1
        tol = 2.0 ** -8 * np.abs(want) + move * (w + np.abs(want)) + 2.0 ** -10 * w + 2.0 ** -20 * vmax
        assert np.all(err <= tol), f"{what} row {b}: {np.max(err - tol):.3e} over"
        rel = np.sqrt((err ** 2).mean(1) / (want ** 2).mean(1))
        assert np.all(rel <= 1e-2 + move[:, 0]), f"{what} row {b}: rel RMS {rel.max():.3e}"


def _one_size(gen, n, size, G, rows, vscales):
    """Keys of one direction, all of one size or half of it (a tile's first is whole), so that scores are +-size or half of
    that; values whose scale differs from tile to tile; heads of either sign."""
    side = math.sqrt(size / SCALE)
    whole = torch.rand(n, generator=gen, device=DEV) < 0.5
    whole[::16] = True
    k = torch.zeros(n, 1, 192, device=DEV)
    k[:, 0, 100] = torch.where(whole, side, side / 2)
    f = torch.tensor(vscales, device=DEV).repeat_interleave(16).repeat(-(-n // (16 * len(vscales))))[:n]
    v = torch.randn(n, 1, 128, generator=gen, device=DEV) * f[:, None, None]
    q = torch.zeros(rows, G, 192, device=DEV)
    q[..., 100] = side * torch.where(torch.rand(rows, G, generator=gen, device=DEV) < 0.5, -1.0, 1.0)
    q[0, 0, 100] = side
    if G > 1:
        q[0, 1, 100] = -side
    return k.bfloat16(), v.bfloat16(), q.bfloat16(), whole.cpu().numpy()


def _check_one_size(got, q, pos, pool, n, whole, what):
    """The keys that a row's largest score is shared by are alike to the last bit, and the others are thousands below: the
    output is their values' mean.  Beside bf16's 2^-8 |o|, a weight's fp16 rounding and the sums, as in _check."""
    _, V, _ = _values(pool, n)
    vmax = np.abs(V).max()
    for b, p in enumerate(pos):
        for h in range(q.shape[1]):
            most = whole[:p + 1] if float(q[b, h, 100]) > 0 else ~whole[:p + 1]
            if not most.any():
                most = ~most
            want, w = V[:p + 1][most].mean(0), np.abs(V[:p + 1][most]).mean(0)
            err = np.abs(got[b, h] - want)
            tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * w + 2.0 ** -20 * vmax
            assert np.all(err <= tol), f"{what} row {b} head {h}: {np.nanmax(err / tol):.3e} of the bound"


@pytest.mark.parametrize("G,rows", [(4, 1), (8, 1), (16, 1), (4, 4), (8, 4), (16, 4)])
@pytest.mark.parametrize("n,most", [(1, 1), (20, 64), (600, 600), (9000, 9000)])
@pytest.mark.parametrize("size", [1e4, 1e5, 1e6, 1e7, 1e8, 1e9, 1e12, 1e20, 1e29])
def test_scores_of_one_size(table, size, n, most, G, rows):
    """Scores of +-size, where the value scales of other tiles are powers of two apart: a reference that held a scale beside
    a score in one fp32 number would lose it."""
    gen = _gen(int(math.log10(size)) + n + G + rows)
    for vscales in ((1.0,), (1e-3, 1.0, 30.0), (1e-30, 1e-28)):
        k, v, q, whole = _one_size(gen, n, size, G, rows, vscales)
        pool = _pool(gen, k, v, table)
        if most > n:
            pool = kvr.Kv8Layout(pool.data, torch.nn.functional.pad(pool.block_table, (0, -(-most // 64) - 1), value=-1))
        pos = [max(n - rows + i, 0) for i in range(rows)]
        got = _decode(q, pos, pool, table, most)
        _check_one_size(got, q, pos, pool, n, whole, f"{size} {vscales}")


@pytest.mark.parametrize("G,rows", [(4, 1), (8, 1), (16, 1), (4, 4), (8, 4), (16, 4)])
@pytest.mark.parametrize("n,most", [(1, 1), (20, 64), (600, 600), (9000, 9000)])
@pytest.mark.parametrize("size", [1e30, 1e31, 1e32, 1e37])
def test_scores_far_below_zero(table, size, n, most, G, rows):
    """Rows whose scores all lie below -1e30, and as far above zero: no finite score stands for a row without keys."""
    test_scores_of_one_size(table, size, n, most, G, rows)


@pytest.mark.parametrize("G,rows", [(4, 1), (8, 1), (16, 1), (16, 4)])
@pytest.mark.parametrize("n", [200, 9000])
@pytest.mark.parametrize("mag", [1e-30, 1.0, 30.0, 300.0, 3e3])
def test_queries_of_any_size(table, mag, n, G, rows):
    """Scores of random keys, up to tens of thousands."""
    gen = _gen(43 + G + n)
    k = torch.randn(n, 1, 192, generator=gen, device=DEV).bfloat16()
    v = torch.randn(n, 1, 128, generator=gen, device=DEV).bfloat16()
    pool = _pool(gen, k, v, table)
    q = (torch.randn(rows, G, 192, generator=gen, device=DEV) * mag).bfloat16()
    pos = [n - rows + i for i in range(rows)]
    _check(_decode(q, pos, pool, table, n), q, pos, pool, n, f"{mag}")


@pytest.mark.parametrize("G,rows", [(8, 1), (16, 1), (8, 4)])
@pytest.mark.parametrize("n", [1500, 8000])
def test_scores_rise_and_fall(table, n, G, rows):
    """Scores that climb along the keys (every tile raises the maximum), that fall by hundreds, one far above the rest at
    either end, and steps up and down between tiles of other value scales."""
    gen = _gen(47 + n)
    u = torch.zeros(192, device=DEV)
    u[64:] = torch.randn(128, generator=gen, device=DEV)
    u /= u.norm()
    steps = torch.randint(-8, 9, (-(-n // 16),), generator=gen, device=DEV).repeat_interleave(16)[:n].cpu() * 25.0
    f = torch.exp2(torch.randint(-40, 41, (-(-n // 16),), generator=gen, device=DEV).float()).repeat_interleave(16)[:n]
    for ramp, scaled in ((torch.linspace(-300, 300, n), False), (torch.linspace(300, -300, n), False),
                         (torch.eye(n)[0] * 400, False), (torch.eye(n)[-1] * 400, False), (steps, True),
                         (torch.linspace(-300, 300, n), True), (torch.linspace(300, -300, n), True)):
        k = (torch.randn(n, 1, 192, generator=gen, device=DEV) * 0.05 + ramp.to(DEV)[:, None, None] * u * 0.5).bfloat16()
        v = torch.randn(n, 1, 128, generator=gen, device=DEV) * (f[:, None, None] if scaled else 1.0)
        pool = _pool(gen, k, v.bfloat16(), table)
        q = (torch.randn(rows, G, 192, generator=gen, device=DEV) * 0.1 + u * 14).bfloat16()
        pos = [n - rows + i for i in range(rows)]
        _check(_decode(q, pos, pool, table, n), q, pos, pool, n)


@pytest.mark.parametrize("G,rows", [(4, 1), (8, 1), (16, 1), (16, 4)])
@pytest.mark.parametrize("n,most", [(1, 1), (40, 64), (600, 600), (9000, 9000)])
@pytest.mark.parametrize("key,query", [(3e38, 3e38), (3e38, 1e25), (1e20, 3e38)])
def test_large_keys_beside_large_queries(table, key, query, n, most, G, rows):
    """Keys and queries so large that the product of their scales is past fp32, in dims that do not meet: all scores are 0
    and the output is the mean of the values."""
    gen = _gen(n + G)
    k = torch.zeros(n, 1, 192, device=DEV)
    k[:, 0, 64:128] = torch.where(torch.rand(n, 64, generator=gen, device=DEV) < 0.5, -key, key)
    q = torch.zeros(rows, G, 192, device=DEV)
    q[..., 128:] = query
    k, q = k.bfloat16(), q.bfloat16()
    v = torch.randn(n, 1, 128, generator=gen, device=DEV).bfloat16()
    pool = _pool(gen, k, v, table)
    if most > n:
        pool = kvr.Kv8Layout(pool.data, torch.nn.functional.pad(pool.block_table, (0, -(-most // 64) - 1), value=-1))
    pos = [max(n - rows + i, 0) for i in range(rows)]
    _check_one_size(_decode(q, pos, pool, table, most), torch.ones_like(q), pos, pool, n, np.ones(n, bool), f"{key} {query}")
