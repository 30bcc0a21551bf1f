"""Values of the 4-bit decode where bounds elsewhere are wide or no other test goes: scores that rise and fall by
hundreds, queries so large that one key takes everything, long shares of small head groups, draft rows on long
contexts, a million keys, sums over very long pieces, several shares a CTA, values so small that their scales are fp16
subnormals, and calls on two streams at once.

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


# -- scores far apart ----------------------------------------------------------------------------------------------------

def _as_held(q):
    """The query as the kernel holds it, for queries whose rotary dims are zero: q * scale * log2(e) in fp32, times the
    power of two that brings a head's largest magnitude to [2^14, 2^15), to fp16 (odd dims after a division by 16).
    In units of log2, fp64."""
    y = q.float() * float(np.float32(SCALE) * np.float32(1.4426950408889634))
    up = torch.exp2(14 - torch.floor(torch.log2(y.abs().amax(-1, keepdim=True).double()))).float()
    div = torch.where(torch.arange(192, device=DEV) % 2 == 1, 16.0, 1.0)
    return (y * up / div).half().double() * div / up.double()


def _check_held(out, q, K, V, km, ks):
    """One row's heads of one KV head against attention with the query as the kernel holds it.  What is left of a score's
    error is fp32: every product of a sum of at most 14 cuts off below 2^-23 of what it adds up (A: codes and minima
    counted apart), and a group's query sum is held to max|y| 2^-15 beside its minimum.  Returns answer and bound."""
    y = _as_held(q)
    S = y @ K.T
    w = torch.exp2(S - S.amax(1, keepdim=True))
    w /= w.sum(1, keepdim=True)
    want, wv = w @ V, w @ V.abs()
    yg = y.abs().unflatten(1, (3, 64)).sum(-1)                                     # [G, 3]
    A = (yg @ (15 * ks + km.abs()).T).amax(1, keepdim=True)
    d = 14 * 2.0 ** -23 * A + 2.0 ** -15 * y.abs().amax(1, keepdim=True) * km.abs().sum(1).amax()
    assert float(d.max()) < 0.02
    tol = 2.0 ** -8 * want.abs() + (torch.exp2(2 * d) - 1) * (wv + want.abs()) + 2.0 ** -10 * (wv + 3 * V.abs().max())
    err = (out.double() - want).abs()
    assert torch.all(err <= tol), f"{float((err - tol).max()):.3e} over"
    return want, tol


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("n", [1500, 6000])
@pytest.mark.parametrize("kind", ["rise", "fall", "first", "last", "saw"])
def test_scores_rise_and_fall_with_their_values(table, tiles, kind, n, G):
    """Scores that climb along the keys (every unit moves the reference), fall by hundreds, stand out at one end or go up
    and down, over one row's pieces (6000 keys: the work line; 1500: a cluster)."""
    gen = _gen(1000 + n + G)
    t = torch.linspace(-1, 1, n, device=DEV)
    ramp = {"rise": 300 * t, "fall": -300 * t, "first": 400.0 * (t == t[0]), "last": 400.0 * (t == t[-1]),
            "saw": 100 * torch.sin(t * 40)}[kind]
    u = torch.zeros(192, device=DEV)
    u[64:] = _randn(gen, 128)
    u /= u.norm()
    k = (_randn(gen, n, 1, 192) * 0.05 + ramp[:, None, None] * u * 0.5).bfloat16()
    v = _randn(gen, n, 1, 128).bfloat16()
    pool = kvr.Kv4Layout.contiguous(1, 1, n)
    _append(pool, k, v, 0, table)
    q = (_randn(gen, 1, G, 192) * 0.1 + u * 14)
    q[..., :64] = 0
    q = q.bfloat16()
    out = kvr.full_attn_decode_kv4(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
    K, V, km, ks = tiles.keys(pool, 0, 0, n)
    want, tol = _check_held(out[0], q[0], K, V, km, ks)
    # the bound can fail: neither zeros nor the keys' mean nor the answer's negative pass it
    for wrong in (torch.zeros_like(want), V.mean(0).expand_as(want), -want):
        assert torch.any((wrong - want).abs() > 4 * tol)
    assert kvr.device_status() == 0


@pytest.mark.parametrize("G", [8, 16])
def test_minima_far_from_zero_under_cancelling_queries(table, tiles, G):
    """Keys around +40 in every dim under queries whose dims of a group add up to next to nothing: the minima's product
    is a large number times a small one."""
    gen = _gen(77 + G)
    n = 5000
    k = _randn(gen, n, 1, 192) + 40
    pool = kvr.Kv4Layout.contiguous(1, 1, n)
    _append(pool, k.bfloat16(), _randn(gen, n, 1, 128).bfloat16(), 0, table)
    q = _randn(gen, 1, G, 192).bfloat16().float()
    q[..., :64] = 0
    for lo in (64, 128):  # bf16 values that cancel in pairs, but for one dim
        q[..., lo + 33:lo + 64] = -q[..., lo + 1:lo + 32].flip(-1)
    q = q.bfloat16()
    out = kvr.full_attn_decode_kv4(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
    _check_held(out[0], q[0], *tiles.keys(pool, 0, 0, n))
    assert kvr.device_status() == 0


@pytest.mark.parametrize("G", [4, 16])
def test_one_key_takes_everything(table, tiles, G):
    """Queries of magnitude 1e4: the best key's logit leads by hundreds (asserted), so its value is the answer, in every
    KV head."""
    gen = _gen(43 + G)
    n, hkv = 200, 2
    pool = kvr.Kv4Layout.contiguous(1, hkv, n)
    _append(pool, _randn(gen, n, hkv, 192).bfloat16(), _randn(gen, n, hkv, 128).bfloat16(), 0, table)
    q = (_randn(gen, 1, hkv * G, 192) * 1e4).bfloat16()
    out = kvr.full_attn_decode_kv4(q, _ints([n - 1], torch.int64), _ints([0], torch.int32), pool, table, SCALE, n)
    for h in range(hkv):
        K, V, _, _ = tiles.keys(pool, 0, h, n)
        x = _rotated(q[0, h * G:(h + 1) * G], table[n - 1])
        top = (x @ K.T * SCALE).topk(2, -1)
        # a score is known to 2^-10 sum |q||k|: the lead has to be out of its reach
        lead = top.values[:, 0] - top.values[:, 1]
        reach = 2 * 2.0 ** -10 * (x.abs() @ K.abs().T).amax(1) * SCALE
        sure = lead > reach + 20
        assert int(sure.sum()) >= G // 2
        want = V[top.indices[:, 0]]
        # one weight, rounded to fp16 in numerator (twice) and sum, and the output's half step; the value's code part
        # and minimum counted apart
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * 4 * V.abs().max()
        err = (out[0, h * G:(h + 1) * G].double() - want).abs()
        assert torch.all((err <= tol)[sure])
    assert kvr.device_status() == 0


# -- forms that long contexts reach --------------------------------------------------------------------------------------

@pytest.mark.parametrize("G", [2, 8])
def test_long_shares_of_small_groups_keep_their_digits(table, tiles, G):
    """Shares of 18,000 keys a CTA in the form for up to 8 heads: sums of codes and minima cancel to a hundredth of their
    size.  The output's own rounding is 2^-8 / sqrt(3) in the mean square at most, everything else is held to 2^-11."""
    gen = _gen(213)
    B, ctx, hkv = 32, 65537, 4
    pool = kvr.Kv4Layout.contiguous(B, hkv, ctx, zero=False)
    for s in range(B):
        k, v = _randn(gen, ctx, hkv, 192), _randn(gen, ctx, hkv, 128)
        k[..., 64:] += 0.5 * _randn(gen, 1, hkv, 128)
        _append(pool, k.bfloat16(), v.bfloat16(), s, table)
    q = _randn(gen, B, hkv * G, 192).bfloat16()
    pos = torch.full((B,), ctx - 1, dtype=torch.int64, device=DEV)
    out = kvr.full_attn_decode_kv4(q, pos, torch.arange(B, dtype=torch.int32, device=DEV), pool, table, SCALE, ctx)
    for b, h in ((0, 0), (13, 2), (31, 1)):
        K, V, _, _ = tiles.keys(pool, b, h, ctx)
        want = torch.softmax(_rotated(q[b, h * G:(h + 1) * G], table[ctx - 1]) @ K.T * SCALE, -1) @ V
        err = (out[b, h * G:(h + 1) * G].double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(err.max()) <= 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -11, float(err.max())


@pytest.mark.parametrize("G", [5, 16])
def test_draft_rows_on_long_contexts(table, tiles, G):
    gen = _gen(31 + G)
    lens, C, hkv = [70, 3000, 9001], 4, 2
    pool = kvr.Kv4Layout.contiguous(3, hkv, max(lens), block_size=32)
    for s, n in enumerate(lens):
        _append(pool, _randn(gen, n, hkv, 192).bfloat16(), _randn(gen, n, hkv, 128).bfloat16(), s, table)
    pos = [n - C + c for n in lens for c in range(C)]
    seq = [s for s in range(len(lens)) for _ in range(C)]
    q = _randn(gen, len(pos), hkv * G, 192).bfloat16()
    assert kvr.full_attn_decode_kv4_workspace_size(len(pos), hkv * G, hkv, max(lens)) > 0  # (not the one-launch form)
    out = kvr.full_attn_decode_kv4(q, _ints(pos, torch.int64), _ints(seq, torch.int32), pool, table, SCALE, max(lens))
    for b, (p, s) in enumerate(zip(pos, seq)):
        for h in range(hkv):
            K, V, _, _ = tiles.keys(pool, s, h, p + 1)
            _check(out[b, h * G:(h + 1) * G], q[b, h * G:(h + 1) * G], p, table[p], K, V, f"row {b} head {h}")
    assert kvr.device_status() == 0


@pytest.mark.parametrize("G", [8, 16])
def test_a_million_keys(table, tiles, G):
    gen = _gen(101 + G)
    ctx, hkv, bs, step = 1000003, 1, 48, 1 << 18
    mb = -(-ctx // bs)
    ids = torch.randperm(mb, generator=gen, device=DEV).to(torch.int32)[None].contiguous()
    pool = kvr.Kv4Layout(torch.empty(mb, hkv, bs // 16, kvr.KV4_TILE, dtype=torch.uint8, device=DEV), ids)
    for lo in range(0, ctx, step):
        m = min(step, ctx - lo)
        _append(pool, _randn(gen, m, hkv, 192).bfloat16(), _randn(gen, m, hkv, 128).bfloat16(), 0, table, lo)
    q = (_randn(gen, 3, hkv * G, 192) * 2).bfloat16()
    pos = [ctx - 1, ctx // 3, 131073]
    out = kvr.full_attn_decode_kv4(q, _ints(pos, torch.int64), _ints([0, 0, 0], torch.int32), pool, table, SCALE, ctx)
    K, V, _, _ = tiles.keys(pool, 0, 0, ctx)
    for b, p in enumerate(pos):
        _check(out[b], q[b], p, table[p], K[:p + 1], V[:p + 1], f"row {b}")
    assert kvr.device_status() == 0


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
