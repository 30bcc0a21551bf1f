"""The operators of the 4-bit KV pool and of the page bookkeeping, in their plain form, with the sizes they are timed at.

A 4-bit pool keeps one full-attention layer's K (192 wide, RoPE applied) and V (128 wide, scaled) as 4-bit codes in
groups of 64 dims, each group with an fp16 scale s and minimum m:  value = m + s * code.  A group's m is its least value
rounded down, s is (greatest - m) / 15 rounded up, and code = clamp(rint((x - m) / s), 0, 15), in fp32.

Sixteen consecutive positions of one KV head form a tile of 2912 bytes:
  bytes    0..1535  K codes  [3 groups][8: position & 7][4: sixteen dims][2: position >> 3][16 codes]
  bytes 1536..2559  V codes  [2 groups][8: eight dims][4: position >> 1 & 3][2: position >> 3][2: four dims]
                             [2: position & 1][4 codes]
  bytes 2560..2655  K scales [3 groups][4: position >> 1 & 3][2: position >> 3][2: position & 1]  fp16
  bytes 2656..2719  V scales [2 groups][4][2][2]  fp16, the same order
  bytes 2720..2783  V minima [2 groups][4][2][2]  fp16, the same order
  bytes 2784..2911  K minima [16 positions][4: three groups, then zero]  fp16
A code pair shares a byte, the lower dim in the lower half.  A pool is [blocks][KV heads][block size / 16][2912] bytes.
"""
import math

import torch

own = False

DQK, DV, DROT, G, TILE = 192, 128, 64, 64, 2912
SCALE = 1.0 / math.sqrt(192.0)
VSCALE = 0.707


def listed():
    return [
        # decode, the smallest real call: one short sequence of the tiny configuration
        dict(name="decode_1x513", op="decode", batch=1, ctx=513, hq=8, hkv=2, block=64, ragged=False, shifted=True),
        # one user at 32K: latency
        dict(name="decode_1x32769", op="decode", batch=1, ctx=32769, hq=64, hkv=4, block=64, ragged=False, shifted=True),
        # a serving batch with contexts of every length, odd pages, eight heads per group
        dict(name="decode_ragged_48", op="decode", batch=48, ctx=65536, hq=32, hkv=4, block=48, ragged=True, shifted=False),
        # the serving batch of the benchmark
        dict(name="decode_64x32769", op="decode", batch=64, ctx=32769, hq=64, hkv=4, block=64, ragged=False, shifted=True),
        # the KV write of one decode step, read back
        dict(name="append_64", op="append", batch=64, rows=1, ctx=32769, hkv=4, block=64, by_slot=False),
        # the KV write of a prefill chunk through a slot map, read back for the chunk's own attention
        dict(name="append_8192", op="append", batch=1, rows=8192, ctx=131072, hkv=4, block=64, by_slot=True),
        # a mixed batch of odd chunks
        dict(name="append_37x1021", op="append", batch=37, rows=1021, ctx=4096, hkv=8, block=16, by_slot=False),
        # a short prefix loaded into bf16 pages before a prompt continues
        dict(name="unpack_3x777", op="unpack", batch=3, rows=777, start=101, hkv=4, block=32),
        # the cached prefix of the benchmark's prefill chunk
        dict(name="unpack_1x122880", op="unpack", batch=1, rows=122880, start=0, hkv=4, block=64),
        # block tables and slot map of one decode step
        dict(name="grow_64x1", op="grow", batch=64, add=1, ctx=32768, block=64),
        # a mixed step: many decodes and some prefill chunks
        dict(name="grow_1000_mixed", op="grow", batch=1000, add=400, ctx=131072, block=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "unpack", "grow"])
    block = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "decode":
        hkv = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 64)
        most = 64 * 32769 * 4 // (batch * hkv)
        return dict(op=op, batch=batch, ctx=_log(rng, 1, min(131072, most)), hq=hkv * rng.choice([1, 3, 7, 8, 13, 16]), hkv=hkv,
                    block=block, ragged=rng.random() < 0.5, shifted=rng.random() < 0.5)
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(2, 32768 // batch))
        return dict(op=op, batch=batch, rows=rows, ctx=max(rows, _log(rng, 512, 8192)), hkv=hkv, block=block, by_slot=rng.random() < 0.5)
    if op == "unpack":
        batch = _log(rng, 1, 32)
        return dict(op=op, batch=batch, rows=_log(rng, 1, 122880 // batch), start=rng.randrange(0, 1000), hkv=rng.choice([1, 2, 4]), block=block)
    batch = _log(rng, 1, 1000)
    return dict(op=op, batch=batch, add=_log(rng, 1, 400), ctx=_log(rng, 1, 131072), block=block)


# -- the 4-bit form, plainly ---------------------------------------------------------------------------------------------

def _step(h, up):
    """The next fp16 value above (up) or below h."""
    b = h.view(torch.int16).to(torch.int32)
    neg = b < 0
    away = torch.where(neg, b + 1, b - 1) if not up else torch.where(neg, b - 1, b + 1)
    zero = (b & 0x7FFF) == 0
    away = torch.where(zero, torch.full_like(b, 1 if up else -32767), away)
    return away.to(torch.int16).view(torch.float16)


def _fp16_down(x):
    h = x.clamp(-65504.0, 65504.0).to(torch.float16)
    return torch.where(h.float() > x, _step(h, False), h)


def _fp16_up(x):
    h = x.clamp(-65504.0, 65504.0).to(torch.float16)
    return torch.where(h.float() < x, _step(h, True), h)


def _quantise(x):
    """x [..., n * 64] fp32 -> codes (uint8), scales and minima [..., n] fp16."""
    g = x.unflatten(-1, (-1, G))
    m = _fp16_down(g.amin(-1))
    s = _fp16_up((g.amax(-1) - m.float()) / torch.full_like(m, 15, dtype=torch.float32))
    step = torch.where(s > 0, s.float(), torch.full_like(s, math.inf, dtype=torch.float32))
    u = torch.round((g - m.float()[..., None]) / step[..., None]).clamp(0, 15).to(torch.uint8)
    return u.flatten(-2), s, m


def _dequantise(u, s, m):
    return (u.unflatten(-1, (-1, G)).float() * s.float()[..., None] + m.float()[..., None]).flatten(-2)


def _pairs(u):
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _codes(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _tiles(ku, ks, km, vu, vs, vm):
    """Token-major codes and scales [..., 16, width] -> tiles [..., 2912]."""
    lead = ku.shape[:-2]
    n = len(lead)
    ax = list(range(n))

    def order(t, shape, perm):
        return t.reshape(*lead, *shape).permute(*ax, *[n + i for i in perm]).reshape(*lead, -1)

    def raw(t):
        return t.contiguous().view(torch.uint8)

    kc = _pairs(order(ku, (2, 8, 3, 4, 16), (2, 1, 3, 0, 4)))
    vc = _pairs(order(vu, (2, 4, 2, 2, 8, 2, 4), (3, 4, 1, 0, 5, 2, 6)))
    kmp = torch.cat([km, torch.zeros_like(km[..., :1])], -1).reshape(*lead, -1)
    return torch.cat([kc, vc, raw(order(ks, (2, 4, 2, 3), (3, 1, 0, 2))), raw(order(vs, (2, 4, 2, 2), (3, 1, 0, 2))),
                      raw(order(vm, (2, 4, 2, 2), (3, 1, 0, 2))), raw(kmp)], -1)


def _values(tiles):
    """Tiles [..., 2912] -> values K [..., 16, 192] and V [..., 16, 128] in fp32."""
    lead = tiles.shape[:-1]
    n = len(lead)
    ax = list(range(n))

    def order(t, shape, perm):
        return t.reshape(*lead, *shape).permute(*ax, *[n + i for i in perm])

    def half(lo, hi):
        return tiles[..., lo:hi].contiguous().view(torch.float16)

    ku = order(_codes(tiles[..., :1536]), (3, 8, 4, 2, 16), (3, 1, 0, 2, 4)).reshape(*lead, 16, DQK)
    vu = order(_codes(tiles[..., 1536:2560]), (2, 8, 4, 2, 2, 2, 4), (3, 2, 5, 0, 1, 4, 6)).reshape(*lead, 16, DV)
    ks = order(half(2560, 2656), (3, 4, 2, 2), (2, 1, 3, 0)).reshape(*lead, 16, 3)
    vs = order(half(2656, 2720), (2, 4, 2, 2), (2, 1, 3, 0)).reshape(*lead, 16, 2)
    vm = order(half(2720, 2784), (2, 4, 2, 2), (2, 1, 3, 0)).reshape(*lead, 16, 2)
    km = half(2784, 2912).reshape(*lead, 16, 4)[..., :3]
    return _dequantise(ku, ks, km), _dequantise(vu, vs, vm)


def _rope(x, cs):
    """Rotate-half RoPE of x [T, heads, 192] on dims 0..63; cs [T, 32, 2] fp32."""
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = x[..., :32], x[..., 32:64]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 64:]], -1)


# -- inputs --------------------------------------------------------------------------------------------------------------

def _table(max_pos, theta=1e7):
    p = torch.arange(max_pos, dtype=torch.float64, device="cuda")
    f = theta ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32.0)
    a = p[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def _pool(gen, blocks, hkv, block, shift):
    """A filled 4-bit pool: keys with a common offset (or none), values of unit variance."""
    data = torch.empty(blocks, hkv, block // 16, TILE, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (hkv * block * (DQK + DV)))
    for lo in range(0, blocks, step):
        n = min(step, blocks - lo)
        shape = (n, hkv, block // 16, 16)
        k = torch.randn(*shape, DQK, generator=gen, device="cuda")
        k[..., DROT:] += shift[None, :, None, None, :]
        v = torch.randn(*shape, DV, generator=gen, device="cuda") * VSCALE
        ku, ks, km = _quantise(k)
        vu, vs, vm = _quantise(v)
        data[lo:lo + n] = _tiles(ku, ks, km, vu, vs, vm)
    return data


def _blocks(gen, need):
    """A block table [len(need), max(need)] of distinct blocks in random order, -1 behind each sequence's own."""
    total = sum(need)
    ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    at = torch.arange(max(need), device="cuda")
    first = n.cumsum(0) - n
    idx = (first[:, None] + at).clamp(max=total - 1)
    return torch.where(at < n[:, None], ids[idx], torch.full_like(idx, -1, dtype=torch.int32)).contiguous(), total


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    op, block = case["op"], case["block"]
    s = dict(op=op, case=case, block=block)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if op == "decode":
        B, ctx, hq, hkv = case["batch"], case["ctx"], case["hq"], case["hkv"]
        if case["ragged"]:
            u = torch.rand(B, generator=gen, device="cuda", dtype=torch.float64)
            lens = torch.exp(u * math.log(ctx)).round().clamp(1, ctx).long().tolist()
        else:
            lens = [ctx] * B
        table, total = _blocks(gen, [-(-n // block) for n in lens])
        # logits of mean -25 and deviation 3 where shifted: q and k lie along one direction, with opposite signs
        u = torch.zeros(hkv, DQK - DROT, device="cuda")
        alpha = beta = 0.0
        if case["shifted"]:
            u = rand(hkv, DQK - DROT)
            u = u / u.norm(dim=1, keepdim=True)
            prod, both = 25 * math.sqrt(DQK), DQK * 8.0
            a, b = math.sqrt(both + 2 * prod), math.sqrt(both - 2 * prod)
            alpha, beta = (a - b) / 2, (a + b) / 2
        s["data"] = _pool(gen, total, hkv, block, -beta * u)
        q = rand(B, hq, DQK)
        q[..., DROT:] += alpha * u.repeat_interleave(hq // hkv, 0)
        s.update(q=q.to(torch.bfloat16), table=table, rope=_table(ctx), max_ctx=ctx,
                 pos=torch.tensor([n - 1 for n in lens], dtype=torch.int64, device="cuda"),
                 seq=torch.arange(B, dtype=torch.int32, device="cuda"))
    elif op == "append":
        B, n, ctx, hkv = case["batch"], case["rows"], case["ctx"], case["hkv"]
        table, total = _blocks(gen, [-(-ctx // block)] * B)
        k, v = rand(B * n, hkv, DQK), rand(B * n, hkv, DV)
        k[..., DROT:] -= 0.8 * rand(1, hkv, DQK - DROT)
        P0 = torch.randint(0, ctx - n + 1, (B,), generator=gen, device="cuda")
        pos = (P0[:, None] + torch.arange(n, device="cuda")).reshape(-1)
        seq = torch.arange(B, device="cuda").repeat_interleave(n)
        s.update(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16), pos=pos, seq=seq.to(torch.int32), P0=P0, table=table,
                 rope=_table(ctx), seqs=torch.arange(B, dtype=torch.int32, device="cuda"),
                 cu=torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda"),
                 slots=table[seq, pos // block].long() * block + pos % block,
                 data=torch.zeros(total, hkv, block // 16, TILE, dtype=torch.uint8, device="cuda"))
    elif op == "unpack":
        B, n, lo, hkv = case["batch"], case["rows"], case["start"], case["hkv"]
        table, total = _blocks(gen, [-(-(lo + n) // block)] * B)
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        s.update(data=_pool(gen, total, hkv, block, 0.8 * rand(hkv, DQK - DROT)), table=table, cu=cu,
                 lo=torch.full((B,), lo, dtype=torch.int64, device="cuda"),
                 seqs=torch.arange(B, dtype=torch.int32, device="cuda"),
                 k=torch.empty(B * n, hkv, DQK, dtype=torch.bfloat16, device="cuda"),
                 v=torch.empty(B * n, hkv, DV, dtype=torch.bfloat16, device="cuda"))
    else:
        B, ctx = case["batch"], case["ctx"]
        lens = torch.exp(torch.rand(B, generator=gen, device="cuda", dtype=torch.float64) * math.log(ctx)).long()
        add = torch.ones(B, dtype=torch.int32, device="cuda")
        if case["add"] > 1:  # a fifth of the requests bring a chunk, some bring nothing
            u = torch.rand(B, 2, generator=gen, device="cuda")
            add = torch.where(u[:, 0] < 0.2, (u[:, 1] * case["add"] + 1).int(), (u[:, 0] < 0.9).int())
        rows = B * case["add"] + 5
        old = (lens + block - 1) // block
        width = -(-(ctx + case["add"]) // block)
        first = old.cumsum(0) - old
        at = torch.arange(width, device="cuda")
        S = B + 3
        held = int(old.sum())
        num = held + B * (case["add"] // block + 2)
        ids = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
        seqs = torch.randperm(S, generator=gen, device="cuda")[:B].to(torch.int32)
        table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        idx = (first[:, None] + at).clamp(max=num - 1)
        table[seqs.long()] = torch.where(at < old[:, None], ids[idx], torch.full_like(idx, -1, dtype=torch.int32))
        free = torch.full((num,), -1, dtype=torch.int32, device="cuda")
        free[:num - held] = ids[held:]

        def ints(n, t):
            return torch.empty(n, dtype=t, device="cuda")

        s.update(lens=lens, add=add, seqs=seqs, table=table, free=free, num=num,
                 count=torch.tensor([num - held], dtype=torch.int32, device="cuda"), left=ints(1, torch.int32),
                 cu=ints(B + 1, torch.int32), pos=ints(rows, torch.int64), rseq=ints(rows, torch.int32),
                 slots=ints(rows, torch.int64))
    return s


# -- one pass ------------------------------------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sinks_kv_ring_gb300 as kvr
    op = s["op"]
    if op == "grow":
        kvr.kv_pages_grow(s["table"], s["num"], s["block"], s["seqs"], s["lens"], s["add"], s["free"], s["count"], s["cu"],
                          s["pos"], s["rseq"], s["slots"], free_count_out=s["left"])
        return dict(table=s["table"], left=s["left"], cu=s["cu"], pos=s["pos"], seq=s["rseq"], slots=s["slots"])
    pool = kvr.Kv4Layout(s["data"], s["table"])
    if op == "decode":
        most = min(s["max_ctx"], pool.max_blocks * pool.block_size)  # ragged: the longest drawn may be shorter than the range's end
        return kvr.full_attn_decode_kv4(s["q"], s["pos"], s["seq"], pool, s["rope"], SCALE, most)
    if op == "append":
        T, hkv = s["k"].shape[:2]
        rows = kvr.LinearLayout.empty(T, hkv)
        if s["case"]["by_slot"]:
            kvr.kv4_append_rope(s["k"], s["v"], s["pos"], None, s["rope"], VSCALE, pool, slots=s["slots"])
        else:
            kvr.kv4_append_rope(s["k"], s["v"], s["pos"], s["seq"], s["rope"], VSCALE, pool)
        kvr.kv4_unpack(pool, s["seqs"], s["P0"], s["cu"], rows)
        return rows.k, rows.v
    kvr.kv4_unpack(pool, s["seqs"], s["lo"], s["cu"], kvr.LinearLayout(s["k"], s["v"]))
    return s["k"], s["v"]


def _run_plain(s):
    op, block = s["op"], s["block"]
    if op == "decode":
        q, pos, seq = s["q"], s["pos"], s["seq"].long()
        B, hq = q.shape[:2]
        hkv = s["data"].shape[1]
        t = s["data"][s["table"][seq].clamp(min=0).long()]                      # [B, blocks, heads, tiles, 2912]
        k, v = _values(t.transpose(1, 2).reshape(B, hkv, -1, TILE))
        k, v = k.flatten(2, 3), v.flatten(2, 3)                                 # [B, heads, keys, width]
        x = _rope(q.float(), s["rope"][pos]).reshape(B, hkv, hq // hkv, DQK)
        logit = torch.matmul(x, k.transpose(2, 3)) * SCALE
        after = torch.arange(k.shape[2], device=q.device) > pos[:, None]
        logit.masked_fill_(after[:, None, None], -math.inf)
        w = torch.exp(logit - logit.amax(-1, keepdim=True))
        o = torch.matmul(w, v) / w.sum(-1, keepdim=True)
        return o.reshape(B, hq, DV).to(torch.bfloat16)
    if op == "append":
        k, v = s["k"].float(), s["v"].float() * VSCALE
        T, hkv = k.shape[:2]
        ku, ks, km = _quantise(_rope(k, s["rope"][s["pos"]]))
        vu, vs, vm = _quantise(v)
        slot = s["slots"] if s["case"]["by_slot"] else s["table"][s["seq"].long(), s["pos"] // block].long() * block + s["pos"] % block
        # one position's bytes at their places of its tile
        place = _places(slot.device)[slot % 16]                                 # [T, 180]
        tile = (slot // block)[:, None] * (hkv * (block // 16)) + torch.arange(hkv, device=slot.device) * (block // 16) + (slot % block // 16)[:, None]
        at = tile[..., None] * TILE + place[:, None]                            # [T, heads, 180]
        flat = s["data"].view(-1)
        flat[at] = torch.cat([_pairs(ku), _pairs(vu)] + [t.contiguous().view(torch.uint8) for t in (ks, vs, vm, km)], -1)
        b = flat[at]
        half = b[..., 160:].contiguous().view(torch.float16)
        k = _dequantise(_codes(b[..., :96]), half[..., :3], half[..., 7:])
        v = _dequantise(_codes(b[..., 96:160]), half[..., 3:5], half[..., 5:7])
        return k.to(torch.bfloat16), v.to(torch.bfloat16)
    if op == "unpack":
        T = s["k"].shape[0]
        row = torch.arange(T, device=s["k"].device)
        i = torch.searchsorted(s["cu"].long(), row, right=True) - 1
        p = s["lo"][i] + row - s["cu"].long()[i]
        blk = s["table"][s["seqs"].long()[i], p // block].long()
        k, v = _values(s["data"])                                               # [blocks, heads, tiles, 16, width]
        k, v = (t.flatten(2, 3)[blk, :, p % block] for t in (k, v))
        s["k"].copy_(k)
        s["v"].copy_(v)
        return s["k"], s["v"]
    lens, add, seqs = s["lens"], s["add"].long(), s["seqs"].long()
    have, want = -(-lens // block), -(-(lens + add) // block)
    need = want - have
    first = need.cumsum(0) - need
    total = need.sum()
    at = torch.arange(s["table"].shape[1], device=lens.device)
    k = first[:, None] + at - have[:, None]
    new = (at >= have[:, None]) & (at < want[:, None])
    n0 = s["count"].long()
    ids = s["free"][(n0 - 1 - k).clamp(0, s["free"].shape[0] - 1)]
    s["table"][seqs] = torch.where(new, ids, s["table"][seqs])
    s["left"].copy_(n0 - total)
    s["cu"][:1] = 0
    s["cu"][1:] = add.cumsum(0)
    row = torch.arange(s["pos"].shape[0], device=lens.device)
    i = (torch.searchsorted(s["cu"].long(), row, right=True) - 1)
    live = row < s["cu"][-1]
    i = i.clamp(max=seqs.shape[0] - 1)
    p = lens[i] + row - s["cu"].long()[i]
    none = torch.full_like(p, -1)
    s["pos"].copy_(torch.where(live, p, none))
    s["rseq"].copy_(torch.where(live, seqs[i], none))
    blk = s["table"][seqs[i], torch.where(live, p // block, torch.zeros_like(p))].long()
    s["slots"].copy_(torch.where(live, blk * block + p % block, none))
    return dict(table=s["table"], left=s["left"], cu=s["cu"], pos=s["pos"], seq=s["rseq"], slots=s["slots"])


def _places(device):
    """Where the 180 bytes of a position lie in its tile: [16, 180] (K codes, V codes, K scales, V scales, V minima, K minima)."""
    r = torch.arange(16, device=device)[:, None]
    b = torch.arange(96, device=device)
    kc = b // 32 * 512 + (r & 7) * 64 + b % 32 // 8 * 16 + (r >> 3) * 8 + b % 8
    b = torch.arange(64, device=device)
    vc = 1536 + b // 32 * 512 + b % 32 // 4 * 64 + (r >> 1 & 3) * 16 + (r >> 3) * 8 + b % 4 // 2 * 4 + (r & 1) * 2 + b % 2
    e = (r >> 1 & 3) * 8 + (r >> 3) * 4 + (r & 1) * 2

    def meta(base, n):
        b = torch.arange(2 * n, device=device)
        return base + b // 2 * 32 + e + b % 2

    return torch.cat([kc, vc, meta(2560, 3), meta(2656, 2), meta(2720, 2), 2784 + r * 8 + torch.arange(6, device=device)], 1)


# -- work, and the definition in 64 bits ---------------------------------------------------------------------------------

def work(case):
    op, B = case["op"], case["batch"]
    if op == "decode":
        ctx = case["ctx"]
        # ragged contexts are log-uniform over 1..ctx: their mean
        mean = (ctx - 1) / math.log(ctx) if case["ragged"] and ctx > 1 else ctx
        keys = B * mean
        return dict(bytes=keys * case["hkv"] * 180 + B * case["hq"] * (DQK + DV) * 2, flops=2.0 * keys * case["hq"] * (DQK + DV))
    if op == "append":  # K/V rows in, their 4-bit form and the values it stands for out
        n = B * case["rows"] * case["hkv"]
        return dict(bytes=n * (640 + 180 + 640), flops=n * 320 * 6.0)
    if op == "unpack":
        n = B * case["rows"] * case["hkv"]
        return dict(bytes=n * (180 + 640), flops=n * 320 * 2.0)
    rows = B * case["add"] + 5  # 20 bytes a row, 16 a request, the table's new blocks
    new = B * (0.2 * case["add"] / 2 + 1) / case["block"] if case["add"] > 1 else B / case["block"]
    return dict(bytes=rows * 20 + B * 20 + new * 8, flops=rows * 4.0)


def exact(case, seed):
    op = case["op"]
    if op == "grow":
        return None
    s = prepare(case, seed)
    dev = s["data"].device
    r = torch.arange(16, device=dev)[:, None]
    d = torch.arange(DQK, device=dev)
    # byte and shift of every (position of a tile, dim)
    kb = (d // 64) * 512 + ((r % 8) * 4 + d % 64 // 16) * 16 + r // 8 * 8 + d % 16 // 2
    e = torch.arange(DV, device=dev)
    vb = 1536 + (e // 64) * 512 + (e % 64 // 8 * 4 + r % 8 // 2) * 16 + r // 8 * 8 + e % 8 // 4 * 4 + r % 2 * 2 + e % 4 // 2
    quad = (r % 8 // 2 * 4 + r // 8 * 2 + r % 2)

    def number(t, at):  # the fp16 at byte offsets `at` of tiles [..., 2912], in 64 bits
        bits = t[..., at].int() | (t[..., at + 1].int() << 8)
        frac, ex = (bits & 1023).double(), ((bits >> 10) & 31).long()
        mag = torch.where(ex == 0, frac * 2.0 ** -24, (1024 + frac) * ((ex + 998) << 52).view(torch.float64))
        return torch.where(bits >= 32768, -mag, mag)

    def values(t):  # tiles [n, 2912] -> [n, 16, 192], [n, 16, 128] in 64 bits
        k = ((t[:, kb] >> (d % 2 * 4).to(torch.uint8)) & 15).double()
        v = ((t[:, vb] >> (e % 2 * 4).to(torch.uint8)) & 15).double()
        ks = number(t, 2560 + (torch.arange(3, device=dev) * 16 + quad) * 2)
        vs = number(t, 2656 + (torch.arange(2, device=dev) * 16 + quad) * 2)
        vm = number(t, 2720 + (torch.arange(2, device=dev) * 16 + quad) * 2)
        km = number(t, 2784 + r * 8 + torch.arange(3, device=dev) * 2)
        return (km.repeat_interleave(64, -1) + ks.repeat_interleave(64, -1) * k, vm.repeat_interleave(64, -1) + vs.repeat_interleave(64, -1) * v)

    block = s["block"]
    if op == "decode":
        B, hq, hkv = case["batch"], case["hq"], case["hkv"]
        out = torch.zeros(B, hq, DV, dtype=torch.float64, device=dev)
        for b in range(B):
            p = int(s["pos"][b])
            ang = s["rope"][p].double()
            q = s["q"][b].double()
            q = torch.cat([q[:, :32] * ang[:, 0] - q[:, 32:64] * ang[:, 1], q[:, 32:64] * ang[:, 0] + q[:, :32] * ang[:, 1], q[:, 64:]], 1)
            blocks = s["table"][b, :p // block + 1].long()
            for h in range(hkv):
                k, v = values(s["data"][blocks, h].reshape(-1, TILE))
                k, v = k.reshape(-1, DQK)[:p + 1], v.reshape(-1, DV)[:p + 1]
                for0 = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                out[b, for0] = torch.softmax(q[for0] @ k.T / math.sqrt(192.0), -1) @ v
        return out
    if op == "unpack":
        n, lo = case["rows"], case["start"]
        ks, vs = [], []
        for b in range(case["batch"]):
            blocks = s["table"][b].long()
            t = s["data"][blocks].transpose(0, 1).reshape(-1, TILE)             # heads first
            parts = [values(t[i:i + 4096]) for i in range(0, t.shape[0], 4096)]
            for which, to in ((0, ks), (1, vs)):
                x = torch.cat([c[which].float() for c in parts]).unflatten(0, (case["hkv"], -1)).flatten(1, 2)
                to.append(x[:, lo:lo + n].transpose(0, 1))
        return torch.cat(ks), torch.cat(vs)
    # append: the quantiser's definition in 64 bits
    k, v = s["k"].double(), s["v"].double() * VSCALE
    a = s["rope"].double()[s["pos"]][:, None]
    k = torch.cat([k[..., :32] * a[..., 0] - k[..., 32:64] * a[..., 1], k[..., 32:64] * a[..., 0] + k[..., :32] * a[..., 1], k[..., 64:]], -1)

    def grid(x, way):  # to the fp16 grid, downwards (way = -1) or upwards (1)
        ex = x.abs().clamp(min=2.0 ** -14).view(torch.int64) >> 52
        ulp = ((ex - 10) << 52).view(torch.float64)
        return torch.floor(x / ulp) * ulp if way < 0 else torch.ceil(x / ulp) * ulp

    def both(x):
        g = x.reshape(*x.shape[:-1], -1, 64)
        lo = grid(g.min(-1).values, -1)
        st = grid((g.max(-1).values - lo) / 15, 1)
        u = torch.round((g - lo[..., None]) / st[..., None]).clamp(0, 15)
        return (lo[..., None] + st[..., None] * u).reshape(x.shape)

    return both(k), both(v)
