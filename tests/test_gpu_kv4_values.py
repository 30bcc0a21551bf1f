"""The 4-bit decode over very long contexts and on two streams at once: sums over long pieces, lines of several shares a
CTA, and values so small that their scales are fp16 subnormals.

The oracle is fp64 on the GPU over the values that the codes stand for, from the format's byte offsets alone."""
import math

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
    return kvr.rope_table(1e7, 1 << 20)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(v, t):
    return torch.tensor(v, dtype=t, device=DEV)


def _append(pool, k, v, seq, table, lo=0, vscale=VS):
    T = k.shape[0]
    kvr.kv4_append_rope(k, v, torch.arange(lo, lo + T, device=DEV), torch.full((T,), seq, dtype=torch.int32, device=DEV),
                        table, vscale, pool)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


class _Tiles:
    """Reads tiles [n, 2912] back to fp64."""

    def __init__(self):
        pl = [o4.places(r) for r in range(16)]
        self.at = [torch.tensor(np.array([p[i] for p in pl]), device=DEV) for i in range(6)]
        self.hi = (torch.arange(192, device=DEV) % 2 * 4).to(torch.uint8)

    def part(self, tiles, codes, scales, minima, n):
        half = lambda a: torch.stack([tiles[:, a], tiles[:, a + 1]], -1).contiguous().view(torch.float16)[..., 0].double()
        u = ((tiles[:, self.at[codes]] >> self.hi[:n]) & 15).double()
        m, s = half(self.at[minima]), half(self.at[scales])
        return ((m.repeat_interleave(64, -1) + s.repeat_interleave(64, -1) * u).flatten(0, 1),
                m.flatten(0, 1), s.flatten(0, 1))

    def keys(self, pool, s, h, n):
        """K, V of positions 0..n-1, and K's minima and scales."""
        tiles = pool.data[pool.block_table[s].long(), h].flatten(0, 1)[:-(-n // 16)]
        K, km, ks = self.part(tiles, 0, 2, 5, 192)
        V, _, _ = self.part(tiles, 1, 3, 4, 128)
        return K[:n], V[:n], km[:n], ks[:n]


@pytest.fixture(scope="module")
def tiles():
    return _Tiles()


def _rotated(q, cs):
    q, c, s = q.double(), cs[:, 0].double(), cs[:, 1].double()
    return torch.cat([q[:, :32] * c - q[:, 32:64] * s, q[:, 32:64] * c + q[:, :32] * s, q[:, 64:]], 1)


def _check(got, q, p, cs, K, V, what="", rel_bar=True):
    """One row's heads of one KV head against fp64, by the bound of the decode's own tests: half a bf16 step of the
    output; 2^-10 sum |q||k| of a score (the rotated q rounded to fp16), which moves a weight by twice that; two
    roundings of a weight and one of their sum, 2^-10 of sum p |v| with code part and minimum counted apart (at most
    3 |v|_max of the group of 64 dims)."""
    x = _rotated(q, cs)
    w = torch.softmax(x @ K.T * SCALE, -1)
    want, wv = w @ V, w @ V.abs()
    a = (x.abs() @ K.abs().T).amax(1, keepdim=True) * SCALE
    vmax = V.abs().unflatten(1, (2, 64)).amax((0, 2)).repeat_interleave(64)
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + 2 * 2.0 ** -10 * a * wv + 2.0 ** -10 * (wv + 3 * vmax)
    assert torch.all(err <= tol), f"{what}: {float((err - tol).max()):.3e} over, {float((err / tol).max()):.2f} of the bound"
    rel = float((err.norm(dim=-1) / want.norm(dim=-1)).max())
    assert not rel_bar or rel <= 1e-2, f"{what}: rel RMS {rel:.3e}"


# -- sums and weights at the ends of their range -------------------------------------------------------------------------

@pytest.mark.parametrize("G", [2, 9])
def test_sums_over_very_long_pieces(tiles, G):
    """2^24 keys a row and a row a CTA: a sum that loses its last bit at every one of some 10^5 products a warp would be
    off by half a percent.  A sequence's blocks are 64 blocks over and over, so the answer is attention over their 65,536
    keys.  Values that are all 1 (scale 0) come out as exactly 1; others (mean 1) are within the output's half step and
    2^-10 for everything else."""
    gen = _gen(7 + G)
    B, nb, bs, times = 460, 64, 1024, 256
    n, ctx = nb * bs, nb * bs * times
    rope = torch.zeros(ctx, 32, 2, device=DEV)
    rope[:, :, 0] = 1
    bt = torch.arange(nb, dtype=torch.int32, device=DEV).repeat(times)[None].contiguous()
    pool = kvr.Kv4Layout(torch.zeros(nb, 1, bs // 16, kvr.KV4_TILE, dtype=torch.uint8, device=DEV), bt)
    v = 1 + _randn(gen, n, 1, 128)
    v[..., :64] = 1
    _append(pool, _randn(gen, n, 1, 192).bfloat16(), v.bfloat16(), 0, rope, vscale=1.0)
    q = _randn(gen, B, G, 192).bfloat16()
    pos = torch.full((B,), ctx - 1, dtype=torch.int64, device=DEV)
    out = kvr.full_attn_decode_kv4(q, pos, torch.zeros(B, dtype=torch.int32, device=DEV), pool, rope, SCALE, ctx)
    K, V, _, _ = tiles.keys(kvr.Kv4Layout(pool.data, bt[:, :nb].contiguous()), 0, 0, n)
    assert kvr.device_status() == 0
    assert bool((out[..., :64] == 1).all()), float((out[..., :64].double() - 1).abs().max())
    for b in (0, 200, 459):
        want = torch.softmax(q[b].double() @ K.T * SCALE, -1) @ V
        err = (out[b].double() - want).abs()
        assert torch.all(err <= (2.0 ** -8 + 2.0 ** -10) * want.abs()), float((err / want.abs()).max())


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("B,long", [(80, 80), (80, 3), (300, 100)])
def test_long_ragged_rows_in_turns(table, tiles, B, long, G):
    """Batches whose longest line gives a CTA several shares, with and without contexts that fill it; rows that cannot be
    served among them; the plan made by the split kernel (80 rows) and by one of its own (300)."""
    gen = _gen(19 + B + long + G)
    nb, bs, ctx = 64, 1024, 1 << 20
    n = nb * bs
    pool = kvr.Kv4Layout(torch.zeros(nb, 1, bs // 16, kvr.KV4_TILE, dtype=torch.uint8, device=DEV),
                         torch.arange(nb, dtype=torch.int32, device=DEV).repeat(ctx // n)[None].contiguous())
    _append(pool, _randn(gen, n, 1, 192).bfloat16(), _randn(gen, n, 1, 128).bfloat16(), 0, table)
    lens = torch.exp(torch.rand(B, generator=gen, device=DEV) * math.log(3000)).long()
    lens[torch.randperm(B, generator=gen, device=DEV)[:long]] = ctx - torch.randint(0, 1000, (long,), generator=gen, device=DEV)
    pos, seq = lens - 1, torch.zeros(B, dtype=torch.int32, device=DEV)
    pos[3], seq[7] = -1, 1
    q = _randn(gen, B, G, 192).bfloat16()
    call = lambda: kvr.full_attn_decode_kv4(q, pos, seq, pool, table, SCALE, ctx)
    out = call()
    assert kvr.device_status() == kvr.DEV_BAD_POS | kvr.DEV_BAD_SEQ
    assert not out[3].any() and not out[7].any()
    assert torch.equal(call(), out)
    kvr.device_status()
    K, V, _, _ = tiles.keys(kvr.Kv4Layout(pool.data, pool.block_table[:, :nb].contiguous()), 0, 0, n)
    for b in [0, 1, 2, B - 1] + sorted(range(8, B), key=lambda i: -int(lens[i]))[:4]:
        p = int(pos[b])
        times = torch.full((n,), (p + 1) // n, dtype=torch.float64, device=DEV)   # how often a key occurs
        times[:(p + 1) % n] += 1
        w = torch.softmax(_rotated(q[b], table[p]) @ K.T * SCALE + times.log(), -1)
        want = w @ V
        # half a step of the output; sums cut off by 2^-12 where they are longest, of sum p |v| in numerator and
        # denominator; a key's weight is off by 2^-10 (two roundings, and its score's, from the query's rounding), alike
        # for its repeats and independent from key to key: three standard deviations of the root of their squares
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -11 * (w @ V.abs()) + 3 * 2.0 ** -10 * (w * w @ (V * V)).sqrt()
        err = (out[b].double() - want).abs()
        assert torch.all(err <= tol), f"row {b} ({p + 1} keys): {float((err / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("small,large", [(1e-5, 1e-5), (2e-6, 2e-6), (1e-5, 1.0), (1e-5, 3e3)])
def test_light_keys_of_small_values_count(table, tiles, G, small, large):
    """A few keys that weigh 2^17 times as much as each of the many others, all of whose values are small (in one group
    of dims or both): the others' part, a few percent of the output, has to be there.  A weight of 2^-17 times a value
    scale of 2^-18 is below fp16."""
    gen = _gen(601 + G)
    B, n = 456, 32768
    u = torch.zeros(192, device=DEV)
    u[64:] = _randn(gen, 128)
    u /= u.norm()
    lead = math.sqrt(17.3 * math.log(2) / SCALE)
    k = _randn(gen, n, 1, 192) * 0.02
    k[:, 0, :64] = 0
    k[torch.arange(4, device=DEV) * 32, 0] = lead * u                            # one in each warp's first unit
    v = _randn(gen, n, 1, 128)
    v[..., :64] *= small
    v[..., 64:] *= large
    pool = kvr.Kv4Layout.contiguous(1, 1, n)
    _append(pool, k.bfloat16(), v.bfloat16(), 0, table, vscale=1.0)
    q = (u * lead).expand(B, G, 192).bfloat16().contiguous()
    pos = torch.full((B,), n - 1, dtype=torch.int64, device=DEV)
    out = kvr.full_attn_decode_kv4(q, pos, torch.zeros(B, dtype=torch.int32, device=DEV), pool, table, SCALE, n)
    K, V, _, _ = tiles.keys(pool, 0, 0, n)
    for b in (0, 311, 455):
        _check(out[b], q[b], n - 1, table[n - 1], K, V, f"row {b}")
    assert kvr.device_status() == 0


# -- two streams ---------------------------------------------------------------------------------------------------------

def test_calls_on_two_streams_at_once(table):
    """Calls that allocate for themselves, in turn on the current stream and on another, with nothing between them: each
    gives what it gives alone."""
    gen = _gen(907)
    n, hkv = 30000, 4
    pool = kvr.Kv4Layout.contiguous(2, hkv, n)
    for s in range(2):
        _append(pool, _randn(gen, n, hkv, 192).bfloat16(), _randn(gen, n, hkv, 128).bfloat16(), s, table)
    qs = [_randn(gen, 8, 16 * hkv, 192).bfloat16() for _ in range(2)]
    pos = [_ints([n - 1 - 900 * i for i in range(8)], torch.int64), _ints([n - 1 - 2100 * i for i in range(8)], torch.int64)]
    seq = _ints([0, 1] * 4, torch.int32)
    call = lambda i, st: kvr.full_attn_decode_kv4(qs[i], pos[i], seq, pool, table, SCALE, n, stream=st)
    want = [call(i, None) for i in range(2)]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    outs = [(i, call(i, other if i else None)) for _ in range(30) for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in outs)
    assert kvr.device_status() == 0
