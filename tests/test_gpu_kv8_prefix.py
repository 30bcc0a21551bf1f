"""A prompt that goes on from a prefix kept in 8 bits: the chunk is appended to the
8-bit pool, the sequence read back into bf16 pages (kv8_unpack), and the bf16 prefill
calls attend over those; then the same with the chunk's own rows in bf16."""
import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle.kv4 import attend

from kvr_cases import SCALE, compare_rows_vec
from test_gpu_kv8 import DEV, VS, _append, _built, _filled, _gen, _ints, _kv, _want_unpacked, table  # noqa: F401

pytestmark = pytest.mark.gpu


def _want(q, P0, k, v, table):
    """fp64 attention of q [C, Hq, 192] at positions P0 .. over bf16 keys and values [n, hkv, .] (rotated, scaled)."""
    hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    K, V, qf = k.double().numpy(), v.double().numpy(), q.float().cpu().numpy()
    ok = np.ones(len(K), bool)
    return np.stack([np.concatenate([attend(qf[i, h * G:(h + 1) * G], P0 + i, K[:, h], V[:, h], ok, table[P0 + i].cpu().numpy(),
                                            SCALE)[0] for h in range(hkv)]) for i in range(len(qf))])


@pytest.mark.parametrize("G,bs", [(16, 64), (8, 48)])
@pytest.mark.parametrize("own", [False, True])
def test_prompt_goes_on_from_a_prefix_in_8_bits(table, own, G, bs):  # noqa: F811
    gen = _gen(G + bs)
    hkv, lens, rows = 2, [5, 100, 700, 0], [40, 1, 130, 33]
    n, most = len(lens), 1024
    pool = _filled(gen, lens, hkv, bs, table, max_ctx=most)
    k, v = _kv(gen, sum(rows), hkv)
    _append(pool, k, v, list(range(n)), lens, rows, table)
    pages = kvr.PagedLayout.contiguous(n, hkv, most, block_size=64)
    pages.k.fill_(float("nan"))
    pages.v.fill_(float("nan"))
    seqs, lo = torch.arange(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV)
    back = lens if own else [a + b for a, b in zip(lens, rows)]
    cu = _ints(np.concatenate([[0], np.cumsum(back)]).tolist(), torch.int32)
    kvr.kv8_unpack(pool, seqs, lo, cu, pages, dst_seqs=seqs, T=sum(back))
    if own:                                             # the chunk itself as it was
        pos = torch.cat([torch.arange(a, a + b, device=DEV) for a, b in zip(lens, rows)])
        of = torch.repeat_interleave(seqs, _ints(rows, torch.int64)).contiguous()
        kvr.kv_ring_append_rope(k, v, pos, of, table, VS, pages)
    q = torch.randn(sum(rows), hkv * G, 192, generator=gen, device=DEV).bfloat16()
    at = np.concatenate([[0], np.cumsum(rows)]).tolist()
    varlen = kvr.full_attn_prefill_varlen(q, _ints(at, torch.int32), _ints(lens, torch.int64), seqs, pages, table, SCALE, most)
    for s in range(n):
        a, b, whole = at[s], at[s + 1], lens[s] + rows[s]
        wk, wv = _want_unpacked(pool, s, 0, whole)
        if own:
            kk = pages.k[pages.block_table[s].long()].transpose(1, 2).flatten(0, 1)[:whole].cpu()
            vv = pages.v[pages.block_table[s].long()].transpose(1, 2).flatten(0, 1)[:whole].cpu()
            assert torch.equal(kk[:lens[s]], wk[:lens[s]]) and torch.equal(vv[:lens[s]], wv[:lens[s]])
            wk, wv = kk, vv
        want = _want(q[a:b], lens[s], wk, wv, table)
        chunk = kvr.full_attn_prefill_chunk(q[a:b].contiguous(), lens[s], s, pages, table, SCALE)
        compare_rows_vec(chunk, want, f"chunk {s}")
        compare_rows_vec(varlen[a:b], want, f"varlen {s}")
    assert kvr.device_status() == 0
