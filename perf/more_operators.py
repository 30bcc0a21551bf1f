"""The operators of the 8-bit KV pool and of page sharing, in their plain form, with the sizes they are timed at.

An 8-bit pool keeps one full-attention layer's K (192 wide, RoPE applied) and V (128 wide, scaled) as signed codes u in
-127..127 with one scale for the K and one for the V of 16 consecutive positions of a KV head: value = s * u.  The scale is
the least bf16 number with 127 s >= |x| for every value x of the positions, u = rint(x / s) in fp32.  Positions are appended
in order: one that asks for a larger scale makes the tile's scale grow, and the codes that are there become
rint(u * old / new).  A row (K or V of one position and head) that is not finite has a bit in a mask and reads as NaN.

Sixteen positions of one KV head form a tile of 5136 bytes, a code stored as u + 128:
  bytes    0..3071  K codes [3: sixty-four dims][16 positions][64]
  bytes 3072..5119  V codes [4: thirty-two dims][8: four dims][4: position >> 1 & 3][4 dims][2: position >> 3][2: position & 1]
  bytes 5120..5135  K scale, V scale (fp32), masks of K and V rows that are not finite (16 bits each), zeros
A pool is [blocks][KV heads][block size / 16][5136] bytes.

Page sharing: refs[b] counts the sequences that hold block b beyond the first.
"""
import math

import torch

own = False

DQK, DV, DROT, TILE = 192, 128, 64, 5136
SCALE = 1.0 / math.sqrt(192.0)
VSCALE = 0.707


def listed():
    return [
        # decode, the smallest real call: one short sequence of the tiny configuration
        dict(name="decode8_1x513", op="decode", batch=1, draft=1, ctx=513, hq=8, hkv=2, block=64, ragged=False, shifted=True),
        # one user at 32K: latency
        dict(name="decode8_1x32769", op="decode", batch=1, draft=1, ctx=32769, hq=64, hkv=4, block=64, ragged=False, shifted=True),
        # draft verification: four tokens of each of 12 sequences, as rows of one call
        dict(name="decode8_draft_12x4", op="decode", batch=12, draft=4, ctx=8195, hq=64, hkv=8, block=64, ragged=True, shifted=True),
        # a serving batch with contexts of every length, odd pages, eight heads per group
        dict(name="decode8_ragged_48", op="decode", batch=48, draft=1, ctx=65536, hq=32, hkv=4, block=48, ragged=True, shifted=False),
        # the serving batch of the benchmark
        dict(name="decode8_64x32769", op="decode", batch=64, draft=1, ctx=32769, hq=64, hkv=4, block=64, ragged=False, shifted=True),
        # the KV write of one decode step into tiles that hold earlier tokens, those tiles read back
        dict(name="append8_64", op="append", batch=64, rows=1, ctx=32769, hkv=4, block=64),
        # the KV write of a prefill chunk, read back for the chunk's own attention
        dict(name="append8_8192", op="append", batch=1, rows=8192, ctx=131072, hkv=4, block=64),
        # a mixed batch of odd chunks
        dict(name="append8_37x1021", op="append", batch=37, rows=1021, ctx=4096, hkv=8, block=16),
        # a beam step of a small model: the old beams freed, the best one forked four ways, partial pages copied
        dict(name="fork_4x513", op="fork", parents=1, each=4, ctx=513, hkv=2, block=64, layers=1, kind="bf16"),
        # parallel samples of a serving batch: 8 of each of 16 prompts, four layers kept in 8 bits
        dict(name="fork_16x8", op="fork", parents=16, each=8, ctx=16384, hkv=4, block=64, layers=4, kind="8bit"),
        # a bf16 pool of one layer shrunk after a burst of requests
        dict(name="compact_1500", op="compact", blocks=1500, used=0.45, seqs=40, hkv=4, block=32, layers=1, kind="bf16"),
        # the pools of three layers in 8 bits, shrunk together
        dict(name="compact_6000", op="compact", blocks=6000, used=0.6, seqs=96, hkv=4, block=64, layers=3, kind="8bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "fork", "compact"])
    block = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "decode":
        hkv = rng.choice([1, 2, 4, 8])
        batch, draft = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        most = 64 * 32769 * 4 // (batch * draft * hkv)
        return dict(op=op, batch=batch, draft=draft, ctx=max(draft, _log(rng, 1, min(131072, most))),
                    hq=hkv * rng.choice([1, 3, 7, 8, 13, 16]), hkv=hkv, block=block, ragged=rng.random() < 0.5,
                    shifted=rng.random() < 0.5)
    if op == "append":
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(2, 32768 // batch))
        return dict(op=op, batch=batch, rows=rows, ctx=max(rows, _log(rng, 512, 8192)), hkv=rng.choice([1, 2, 4, 8]), block=block)
    hkv, layers, kind = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 5]), rng.choice(["bf16", "8bit", "4bit"])
    if op == "fork":
        parents = _log(rng, 1, 32)
        return dict(op=op, parents=parents, each=_log(rng, 1, 128 // parents), ctx=_log(rng, 1, 65536 // (parents * layers)), hkv=hkv,
                    block=block, layers=layers, kind=kind)
    each = hkv * block * layers  # positions and heads of a block in all layers
    return dict(op=op, blocks=_log(rng, 8, min(50000, 1500000 // each)), used=rng.uniform(0.05, 0.95), seqs=_log(rng, 1, 200),
                hkv=hkv, block=block, layers=layers, kind=kind)


# -- the 8-bit form, plainly ---------------------------------------------------------------------------------------------

def _least_scale(a):
    """The least bf16 number s with 127 s >= a, as fp32."""
    q = a / torch.full_like(a, 127.0)
    s = ((q.view(torch.int32) + 0xFFFF) & -0x10000)
    s = torch.where(s.view(torch.float32) * 127.0 < a, s + 0x10000, s)
    return s.view(torch.float32)


def _codes(x, s):
    """rint(x / s), 0 where s is 0."""
    q = x / torch.where(s > 0, s, torch.full_like(s, math.inf))
    return torch.round(q).clamp(-127, 127)


def _tiles(ku, vu, ks, vs, kbad, vbad):
    """Codes [..., 16, width], scales and masks [...] -> tiles [..., 5136]."""
    lead = ku.shape[:-2]
    n = len(lead)
    ax = list(range(n))
    k = (ku + 128).to(torch.uint8).reshape(*lead, 16, 3, 64).permute(*ax, n + 1, n, n + 2).reshape(*lead, 3072)
    v = (vu + 128).to(torch.uint8).reshape(*lead, 2, 4, 2, 4, 8, 4).permute(*ax, *[n + i for i in (3, 4, 1, 5, 0, 2)]).reshape(*lead, 2048)
    tail = torch.zeros(*lead, 4, dtype=torch.int32, device=ku.device)
    tail[..., 0] = ks.view(torch.int32)
    tail[..., 1] = vs.view(torch.int32)
    tail[..., 2] = kbad | (vbad << 16)
    return torch.cat([k, v, tail.view(torch.uint8)], -1)


def _parts(tiles):
    """Tiles [..., 5136] -> codes K [..., 16, 192] and V [..., 16, 128] in fp32, scales and masks [...]."""
    lead = tiles.shape[:-1]
    n = len(lead)
    ax = list(range(n))
    ku = tiles[..., :3072].reshape(*lead, 3, 16, 64).permute(*ax, n + 1, n, n + 2).reshape(*lead, 16, DQK)
    vu = tiles[..., 3072:5120].reshape(*lead, 4, 8, 4, 4, 2, 2).permute(*ax, *[n + i for i in (4, 2, 5, 0, 1, 3)]).reshape(*lead, 16, DV)
    tail = tiles[..., 5120:].contiguous().view(torch.int32)
    masks = tail[..., 2]
    return (ku.float() - 128, vu.float() - 128, tail[..., 0].contiguous().view(torch.float32),
            tail[..., 1].contiguous().view(torch.float32), masks & 0xFFFF, (masks >> 16) & 0xFFFF)


def _values(tiles):
    ku, vu, ks, vs, kb, vb = _parts(tiles)
    bit = torch.arange(16, device=tiles.device)
    k, v = ku * ks[..., None, None], vu * vs[..., None, None]
    k.masked_fill_(((kb[..., None] >> bit) & 1 > 0)[..., None], math.nan)
    v.masked_fill_(((vb[..., None] >> bit) & 1 > 0)[..., None], math.nan)
    return k, v


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
    """A filled 8-bit pool: keys with a common offset (or none), values of unit variance."""
    data = torch.empty(blocks, hkv, block // 16, TILE, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (hkv * block * (DQK + DV)))
    for lo in range(0, blocks, step):
        n = min(step, blocks - lo)
        shape = (n, hkv, block // 16, 16)
        k = torch.randn(*shape, DQK, generator=gen, device="cuda")
        k[..., DROT:] += shift[None, :, None, None, :]
        v = torch.randn(*shape, DV, generator=gen, device="cuda") * VSCALE
        ks, vs = _least_scale(k.abs().amax((-1, -2))), _least_scale(v.abs().amax((-1, -2)))
        none = torch.zeros_like(ks, dtype=torch.int32)
        data[lo:lo + n] = _tiles(_codes(k, ks[..., None, None]), _codes(v, vs[..., None, None]), ks, vs, none, none)
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


def _layer_pools(gen, kind, layers, blocks, hkv, block):
    """Each layer's arrays [blocks, ...]: what a page copy moves is bytes, so any values do."""
    out = []
    for _ in range(layers):
        if kind == "bf16":
            out.append([torch.randn(blocks, hkv, block, d, generator=gen, device="cuda", dtype=torch.bfloat16) for d in (DQK, DV)])
        else:
            tile = TILE if kind == "8bit" else 2912
            out.append([torch.randint(0, 256, (blocks, hkv, block // 16, tile), generator=gen, device="cuda", dtype=torch.uint8)])
    return out


def _ints(n, t):
    return torch.full((n,), -1, dtype=t, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    op, block = case["op"], case["block"]
    s = dict(op=op, case=case, block=block)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if op == "decode":
        B, C, ctx, hq, hkv = case["batch"], case["draft"], case["ctx"], case["hq"], case["hkv"]
        if case["ragged"]:
            u = torch.rand(B, generator=gen, device="cuda", dtype=torch.float64)
            lens = torch.exp(u * math.log(ctx)).round().clamp(C, ctx).long().tolist()
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
        q = rand(B * C, hq, DQK)
        q[..., DROT:] += alpha * u.repeat_interleave(hq // hkv, 0)
        pos = torch.tensor(lens, dtype=torch.int64, device="cuda")[:, None] - C + torch.arange(C, device="cuda")
        s.update(q=q.to(torch.bfloat16), table=table, rope=_table(ctx), max_ctx=ctx, pos=pos.reshape(-1).contiguous(),
                 seq=torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(C))
    elif op == "append":
        B, n, ctx, hkv = case["batch"], case["rows"], case["ctx"], case["hkv"]
        table, total = _blocks(gen, [-(-ctx // block)] * B)
        shift = -0.8 * rand(hkv, DQK - DROT)
        k, v = rand(B * n, hkv, DQK), rand(B * n, hkv, DV)
        k[..., DROT:] += shift
        # every place in a tile to start from, each case's own
        r0 = ((torch.arange(B, device="cuda") + n) * 7 % 16).clamp(max=ctx - n)
        P0 = r0 + 16 * (torch.rand(B, generator=gen, device="cuda", dtype=torch.float64) * ((ctx - n - r0) // 16 + 1)).long()
        # what is read back: the chunks, and the tokens that share their first tiles
        back = (P0 % 16 + n).cumsum(0)
        s.update(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16), P0=P0, table=table, rope=_table(ctx),
                 seqs=torch.arange(B, dtype=torch.int32, device="cuda"),
                 cu=torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda"), lo=P0 // 16 * 16,
                 back=torch.cat([torch.zeros_like(back[:1]), back]).to(torch.int32), total=int(back[-1]),
                 data=_pool(gen, total, hkv, block, shift))
    elif op == "fork":
        # beams of the step before hold their parents' whole blocks and a last block of their own
        Pn, each, hkv = case["parents"], case["each"], case["hkv"]
        n = Pn * each
        # prompts of every length up to ctx, evenly over the logarithm
        u = (torch.randperm(Pn, generator=gen, device="cuda").double() + 0.9) / Pn
        lens = torch.exp(u * math.log(case["ctx"])).round().long().clamp(min=1)
        held = -(-lens // block)
        width = -(-case["ctx"] // block) + 1
        first = held.cumsum(0) - held
        used = int(held.sum())
        num = used + 2 * n + 7
        ids = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
        at = torch.arange(width, device="cuda")
        rows = torch.randperm(Pn + n, generator=gen, device="cuda").to(torch.int32)
        src, dst = rows[:Pn].repeat_interleave(each).contiguous(), rows[Pn:].contiguous()
        plens = lens.repeat_interleave(each).contiguous()
        table = torch.full((Pn + n, width), -1, dtype=torch.int32, device="cuda")
        table[rows[:Pn].long()] = torch.where(at < held[:, None], ids[(first[:, None] + at).clamp(max=num - 1)], table[:Pn])
        whole, part = plens // block, plens % block > 0
        beams = torch.where(at < whole[:, None], table[src.long()], -1)
        mine = used + torch.arange(n, device="cuda")
        beams = torch.where((at == whole[:, None]) & part[:, None], ids[mine][:, None], beams)
        table[dst.long()] = beams
        refs = torch.zeros(num, dtype=torch.int32, device="cuda")
        hold = (at < whole[:, None]).reshape(-1)
        refs.index_add_(0, table[src.long()].reshape(-1).clamp(min=0).long(), hold.int())
        free = _ints(num, torch.int32)
        spare = torch.cat([ids[mine][~part], ids[used + n:]]).sort().values
        free[:spare.shape[0]] = spare
        s.update(table=table, refs=refs, src=src, dst=dst, lens=plens, num=num, free=free,
                 count=torch.tensor([spare.shape[0]], dtype=torch.int32, device="cuda"), csrc=_ints(n, torch.int32), cdst=_ints(n, torch.int32),
                 pairs=_ints(1, torch.int32), pools=_layer_pools(gen, case["kind"], case["layers"], num, hkv, block))
    else:
        num, S = case["blocks"], case["seqs"]
        used = max(1, min(num - 1, int(num * case["used"])))
        ids = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
        # short and long sequences: lengths from one share to S shares
        cut = (torch.arange(1, S + 1, device="cuda", dtype=torch.float64).cumsum(0) * (used / (S * (S + 1) / 2))).round().long()
        held = torch.diff(cut, prepend=cut.new_zeros(1))[torch.randperm(S, generator=gen, device="cuda")]
        edge = torch.cat([cut.new_zeros(1), held.cumsum(0)])
        width = int(held.max()) + 1
        at = torch.arange(width, device="cuda")
        table = torch.where(at < held[:, None], ids[(edge[:-1, None] + at).clamp(max=num - 1)], -1).to(torch.int32)
        refs = torch.zeros(num, dtype=torch.int32, device="cuda")
        # a tenth of the sequences share the first blocks of the one before them
        for i in range(10, S, 10):
            m = int(min(held[i], held[i - 1])) // 2
            table[i, :m] = table[i - 1, :m]
            refs[table[i, :m].long()] += 1
        table = table[torch.randperm(S, generator=gen, device="cuda")].contiguous()
        there = torch.zeros(num, dtype=torch.bool, device="cuda")
        there[table[table >= 0].long()] = True
        left = (~there).nonzero().flatten().to(torch.int32)
        left = left[torch.randperm(left.shape[0], generator=gen, device="cuda")]
        free = _ints(num, torch.int32)
        free[:left.shape[0]] = left
        s.update(table=table, refs=refs, num=num, free=free, count=torch.tensor([left.shape[0]], dtype=torch.int32, device="cuda"),
                 table2=torch.empty_like(table), refs2=torch.empty_like(refs), free2=torch.full_like(free, -1),
                 csrc=_ints(num, torch.int32), cdst=_ints(num, torch.int32), pairs=_ints(1, torch.int32),
                 pools=_layer_pools(gen, case["kind"], case["layers"], num, case["hkv"], block))
    return s


# -- one pass ------------------------------------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sinks_kv_ring_gb300 as kvr
    op = s["op"]
    if op == "decode":
        pool = kvr.Kv8Layout(s["data"], s["table"])
        most = min(s["max_ctx"], pool.max_blocks * pool.block_size)  # ragged: the longest drawn may be shorter than the range's end
        return kvr.full_attn_decode_kv8(s["q"], s["pos"], s["seq"], pool, s["rope"], SCALE, most)
    if op == "append":
        pool = kvr.Kv8Layout(s["data"], s["table"])
        rows = kvr.LinearLayout.empty(s["total"], pool.num_kv_heads)
        kvr.kv8_append_rope(s["k"], s["v"], s["cu"], s["P0"], s["seqs"], s["rope"], VSCALE, pool)
        kvr.kv8_unpack(pool, s["seqs"], s["lo"], s["back"], rows)
        return rows.k, rows.v
    kind = s["case"]["kind"]
    make = {"bf16": kvr.PagedLayout, "8bit": kvr.Kv8Layout, "4bit": kvr.Kv4Layout}[kind]
    pools = [make(*a, s["table"]) for a in s["pools"]]
    if op == "fork":
        kvr.kv_pages_free(s["table"], s["num"], s["block"], s["refs"], s["dst"], s["free"], s["count"])
        kvr.kv_pages_fork(s["table"], s["num"], s["block"], s["refs"], s["src"], s["dst"], s["lens"], s["free"], s["count"],
                          s["csrc"], s["cdst"], s["pairs"])
    else:
        kvr.kv_pages_compact(s["table"], s["num"], s["refs"], s["free"], s["count"], s["csrc"], s["cdst"], s["pairs"],
                             table_out=s["table2"], refs_out=s["refs2"], free_ids_out=s["free2"])
    kvr.kv_pages_copy(pools, s["csrc"], s["cdst"], s["pairs"])
    return _state(s)


def _state(s):
    """What the page operators leave: tables, counts, the free list, and the pools' bytes."""
    to = "" if s["op"] == "fork" else "2"
    return dict(table=s["table" + to], refs=s["refs" + to], count=s["count"], pairs=s["pairs"], free=s["free" + to],
                pools=[a for p in s["pools"] for a in p])


def _run_plain(s):
    op, block = s["op"], s["block"]
    if op == "decode":
        q, pos, seq = s["q"], s["pos"], s["seq"].long()
        C = s["case"]["draft"]
        R, hq = q.shape[:2]
        hkv = s["data"].shape[1]
        t = s["data"][s["table"][seq[::C]].clamp(min=0).long()]                 # [B, blocks, heads, tiles, 5136]
        B = t.shape[0]
        k, v = _values(t.transpose(1, 2).reshape(B, hkv, -1, TILE))
        k, v = k.flatten(2, 3), v.flatten(2, 3)                                 # [B, heads, keys, width]
        x = _rope(q.float(), s["rope"][pos]).reshape(B, C, hkv, hq // hkv, DQK)
        x = x.transpose(1, 2).reshape(B, hkv, -1, DQK)                          # rows: draft token, then head of the group
        logit = torch.matmul(x, k.transpose(2, 3)) * SCALE
        after = torch.arange(k.shape[2], device=q.device) > pos.reshape(B, C, 1)
        logit.masked_fill_(after.repeat_interleave(hq // hkv, 1)[:, None], -math.inf)
        w = torch.exp(logit - logit.amax(-1, keepdim=True))
        o = torch.matmul(w, v) / w.sum(-1, keepdim=True)
        return o.reshape(B, hkv, C, -1, DV).transpose(1, 2).reshape(R, hq, DV).to(torch.bfloat16)
    if op == "append":
        return _append_plain(s)
    if op == "fork":
        return _fork_plain(s)
    return _compact_plain(s)


def _append_plain(s):
    block, P0, n = s["block"], s["P0"], s["case"]["rows"]
    B, hkv = P0.shape[0], s["k"].shape[1]
    dev = P0.device
    pos = (P0[:, None] + torch.arange(n, device=dev)).reshape(-1)
    k, v = _rope(s["k"].float(), s["rope"][pos]), s["v"].float() * VSCALE
    # the chunks' rows at their places of the tiles that they touch
    nt = (n + 30) // 16
    r0 = P0 % 16
    at = (torch.arange(B, device=dev)[:, None] * nt * 16 + r0[:, None] + torch.arange(n, device=dev)).reshape(-1)

    def lay(x):
        y = torch.zeros(B * nt * 16, hkv, x.shape[-1], device=dev)
        y[at] = x
        return y.reshape(B, nt, 16, hkv, -1).transpose(2, 3)                    # [B, tiles, heads, 16, width]

    row = torch.arange(nt * 16, device=dev).reshape(nt, 16)
    new = (row >= r0[:, None, None]) & (row < r0[:, None, None] + n)            # [B, tiles, 16]
    live = row < r0[:, None, None]
    some = new.any(-1)
    tile = P0[:, None] // 16 + torch.arange(nt, device=dev)
    per = block // 16
    blk = s["table"].gather(1, (tile // per).clamp(max=s["table"].shape[1] - 1)).long()
    idx = ((blk[..., None] * hkv + torch.arange(hkv, device=dev)) * per + (tile % per)[..., None])  # [B, tiles, heads]
    flat = s["data"].view(-1, TILE)
    idx = torch.where(some[..., None], idx, idx[:, :1])                         # (a tile behind the chunk's last: not written)
    old = _parts(flat[idx])
    bit = 1 << torch.arange(16, device=dev)
    res = []
    for x, u, so, bad in ((lay(k), old[0], old[2], old[4]), (lay(v), old[1], old[3], old[5])):
        odd = ~torch.isfinite(x).all(-1)                                        # [B, tiles, heads, 16]
        x = torch.where(odd[..., None], torch.zeros_like(x), x)
        so = torch.where(live.any(-1)[..., None], so, torch.zeros_like(so))
        sn = torch.maximum(so, _least_scale(x.abs().amax((-1, -2))))
        keep = live[:, :, None, :, None]
        c = torch.where(keep, _codes(u * so[..., None, None], sn[..., None, None]), _codes(x, sn[..., None, None]))
        mask = ((odd & new[:, :, None]) * bit).sum(-1) + (((bad[..., None] & bit) > 0) & live[:, :, None]).mul(bit).sum(-1)
        res += [(c, sn, mask.to(torch.int32))]
    (kc, ks, km), (vc, vs, vm) = res
    out = _tiles(kc, vc, ks, vs, km, vm)
    # (an index that stands twice is the chunk's first tile, with the same bytes)
    out = torch.where(some[..., None, None], out, out[:, :1])
    flat[idx] = out
    k, v = _values(out)
    i = torch.searchsorted(s["back"].long(), torch.arange(s["total"], device=dev), right=True) - 1
    at = i * nt * 16 + torch.arange(s["total"], device=dev) - s["back"].long()[i]
    return tuple(t.transpose(2, 3).reshape(B * nt * 16, hkv, -1)[at].to(torch.bfloat16) for t in (k, v))


def _fork_plain(s):
    table, refs, free, block = s["table"], s["refs"], s["free"], s["block"]
    src, dst, lens = s["src"].long(), s["dst"].long(), s["lens"]
    num = s["num"]
    # free: every holder gives its blocks up, those without a holder go to the list in ascending order
    ids = table[dst]
    has = ids >= 0
    refs.index_add_(0, ids.clamp(min=0).reshape(-1).long(), -has.reshape(-1).int())
    table[dst] = -1
    dead = refs < 0
    rank = dead.cumsum(0) - 1
    into = torch.where(dead, s["count"] + rank, num)
    more = torch.cat([free, free.new_zeros(1)])
    more[into] = torch.arange(num, device=free.device, dtype=torch.int32)
    free.copy_(more[:num])
    refs.clamp_(min=0)
    s["count"] += dead.sum()
    # fork
    width = table.shape[1]
    at = torch.arange(width, device=free.device)
    whole, part = lens // block, lens % block > 0
    ids = table[src]
    share = at < whole[:, None]
    k = part.long().cumsum(0) - 1
    fresh = free[(s["count"].long() - 1 - k).clamp(0, num - 1)]
    tail = (at == whole[:, None]) & part[:, None]
    table[dst] = torch.where(share, ids, torch.where(tail, fresh[:, None], -1))
    refs.index_add_(0, ids.clamp(min=0).reshape(-1).long(), share.reshape(-1).int())
    n = part.shape[0]
    to = torch.where(part, k, n)
    last = ids.gather(1, whole.clamp(max=width - 1)[:, None])[:, 0]
    for name, x in (("csrc", last), ("cdst", fresh)):
        y = torch.cat([s[name], s[name].new_zeros(1)])
        y[to] = x
        s[name].copy_(y[:n])
    s["pairs"].copy_(part.sum().to(torch.int32))
    s["count"] -= s["pairs"]
    _copy_plain(s, n)
    return _state(s)


def _copy_plain(s, most):
    """The pairs' blocks; a pair past the last is the first one again (or block 0 onto itself)."""
    live = torch.arange(most, device=s["csrc"].device) < s["pairs"]
    a, b = (torch.where(live, s[x][:most], s[x][:1]).clamp(min=0).long() for x in ("csrc", "cdst"))
    for p in s["pools"]:
        for x in p:
            x[b] = x[a]


def _compact_plain(s):
    num, free, table = s["num"], s["free"], s["table"]
    dev = free.device
    at = torch.arange(num, device=dev)
    gone = torch.zeros(num + 1, dtype=torch.bool, device=dev)
    gone[torch.where(at < s["count"], free, num).long()] = True
    gone = gone[:num]
    used = num - s["count"].long()
    hole, mover = gone & (at < used), ~gone & (at >= used)
    # the k-th block from `used` on that holds something takes the k-th free place below it
    rank_h, rank_m = hole.cumsum(0) - 1, mover.cumsum(0) - 1
    for name, m, rank in (("csrc", mover, rank_m), ("cdst", hole, rank_h)):
        y = torch.cat([s[name], s[name].new_zeros(1)])
        y[torch.where(m, rank, num)] = at.int()
        s[name].copy_(y[:num])
    s["pairs"].copy_(mover.sum().to(torch.int32))
    new = torch.where(mover, s["cdst"][rank_m.clamp(min=0)].long(), at)
    s["table2"].copy_(torch.where(table >= 0, new[table.clamp(min=0).long()], -1))
    refs = torch.cat([torch.zeros_like(s["refs"]), s["refs"].new_zeros(1)])
    refs[torch.where(gone, num, new)] = s["refs"]
    s["refs2"].copy_(refs[:num])
    s["free2"].copy_(torch.where(at < s["count"], num - 1 - at, -1))
    _copy_plain(s, num // 2 + 1)  # (no more than half of the blocks can have to move)
    return _state(s)


# -- work, and the definition in 64 bits ---------------------------------------------------------------------------------

def _block_bytes(case):
    each = {"bf16": 640, "8bit": TILE / 16, "4bit": 182}[case["kind"]]
    return each * case["hkv"] * case["block"] * case["layers"]


def work(case):
    op = case["op"]
    if op == "decode":
        ctx = case["ctx"]
        # ragged contexts are log-uniform over 1..ctx: their mean
        mean = (ctx - 1) / math.log(ctx) if case["ragged"] and ctx > 1 else ctx
        keys, rows = case["batch"] * mean, case["batch"] * case["draft"]
        return dict(bytes=keys * case["hkv"] * TILE / 16 + rows * case["hq"] * (DQK + DV) * 2,
                    flops=2.0 * keys * case["draft"] * case["hq"] * (DQK + DV))
    if op == "append":  # K/V rows in, their 8-bit form and the values it stands for out
        n = case["batch"] * case["rows"] * case["hkv"]
        return dict(bytes=n * (640 + 321 + 640), flops=n * 320 * 6.0)
    if op == "fork":
        n = case["parents"] * case["each"]
        ctx = case["ctx"]
        mean = (ctx - 1) / math.log(ctx) if ctx > 1 else ctx
        held = n * (mean / case["block"] + 1)  # table entries freed and made again, counts with them
        return dict(bytes=held * 24 + n * (16 + 2 * _block_bytes(case)), flops=held * 2.0)
    moved = case["blocks"] * case["used"] * (1 - case["used"])
    return dict(bytes=case["blocks"] * 24 + moved * 2 * _block_bytes(case), flops=case["blocks"] * 4.0)


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    dev = s["data"].device
    r = torch.arange(16, device=dev)[:, None]
    d, e = torch.arange(DQK, device=dev), torch.arange(DV, device=dev)
    kb = d // 64 * 1024 + r * 64 + d % 64
    vb = 3072 + e // 32 * 512 + (e % 32 // 4 * 4 + r % 8 // 2) * 16 + e % 4 * 4 + r // 8 * 2 + r % 2

    def number(t, at):  # the fp32 at byte `at` of tiles [n, 5136], in 64 bits
        w = sum(t[:, at + i].long() << (8 * i) for i in range(4))
        mag = (2 ** 23 * ((w >> 23 & 255) > 0) + (w & 0x7FFFFF)).double() * torch.exp2(((w >> 23 & 255).clamp(min=1) - 150).double())
        return torch.where(w >> 31 > 0, -mag, mag)[:, None, None]

    def values(t):  # tiles [n, 5136] -> [n, 16, 192], [n, 16, 128] in 64 bits
        return number(t, 5120) * (t[:, kb].double() - 128), number(t, 5124) * (t[:, vb].double() - 128)

    block = s["block"]
    if op == "decode":
        B, C, hq, hkv = case["batch"], case["draft"], case["hq"], case["hkv"]
        G = hq // hkv
        out = torch.zeros(B * C, hq, DV, dtype=torch.float64, device=dev)
        for b in range(B):
            last = int(s["pos"][b * C + C - 1])
            blocks = s["table"][b, :last // block + 1].long()
            for h in range(hkv):
                k, v = values(s["data"][blocks, h].reshape(-1, TILE))
                k, v = k.reshape(-1, DQK), v.reshape(-1, DV)
                for c in range(C):
                    p = int(s["pos"][b * C + c])
                    ang = s["rope"][p].double()
                    q = s["q"][b * C + c, h * G:(h + 1) * G].double()
                    q = torch.cat([q[:, :32] * ang[:, 0] - q[:, 32:64] * ang[:, 1], q[:, 32:64] * ang[:, 0] + q[:, :32] * ang[:, 1], q[:, 64:]], 1)
                    out[b * C + c, h * G:(h + 1) * G] = torch.softmax(q @ k[:p + 1].T / math.sqrt(192.0), -1) @ v[:p + 1]
        return out
    # append: tile by tile of each chunk
    n, hkv = case["rows"], case["hkv"]
    a = s["rope"].double()
    ks, vs = [], []

    def scale(x):  # the least 8-bit-significand number s with 127 s >= max |x| of [heads, rows, width]
        m = x.abs().amax((-1, -2)) / 127
        ex = torch.floor(torch.log2(m.clamp(min=1e-300)))
        ex = torch.where(torch.exp2(ex) > m, ex - 1, ex)
        ulp = torch.exp2(ex - 7)
        return torch.where(m > 0, torch.ceil(m / ulp) * ulp, 0.0)[:, None, None]

    def held(x, sc):
        return sc * torch.round(x / torch.where(sc > 0, sc, 1.0)).clamp(-127, 127)

    starts = s["P0"].tolist()
    table = s["table"].tolist()
    for b in range(case["batch"]):
        P = starts[b]
        p = torch.arange(P, P + n, device=dev)
        k, v = s["k"][b * n:(b + 1) * n].double(), s["v"][b * n:(b + 1) * n].double() * VSCALE
        c, sn = a[p][:, None, :, 0], a[p][:, None, :, 1]
        k = torch.cat([k[..., :32] * c - k[..., 32:64] * sn, k[..., 32:64] * c + k[..., :32] * sn, k[..., 64:]], -1)
        t0 = P // 16
        for which, x, to in ((0, k, ks), (1, v, vs)):
            x = x.transpose(0, 1)
            head = min(16 - P % 16, n)
            got = []
            if P % 16:
                old = s["data"][table[b][t0 * 16 // block], :, t0 % (block // 16)]
                so = number(old, 5120 + 4 * which)
                sc = torch.maximum(so, scale(x[:, :head]))
                got += [held(values(old)[which][:, :P % 16], sc), held(x[:, :head], sc)]
                x = x[:, head:]
            m = x.shape[1] // 16 * 16
            if m:
                y = x[:, :m].reshape(hkv * (m // 16), 16, -1)
                got += [held(y, scale(y)).reshape(hkv, m, -1)]
            if x.shape[1] > m:
                got += [held(x[:, m:], scale(x[:, m:]))]
            to.append(torch.cat(got, 1).transpose(0, 1))
    return torch.cat(ks), torch.cat(vs)
