"""Which pools and tensors the calls over quantised pools take and refuse, without a GPU
(the library is a recorder, as in test_binding_cpu)."""
import pytest
import torch

import sinks_kv_ring_gb300 as kvr

from test_binding_cpu import rec  # noqa: F401

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _z(dtype, *shape):
    return torch.zeros(*shape, dtype=dtype)


def _pools():
    make = [lambda cls=cls: cls.contiguous(3, 2, 100, block_size=32, device="cpu") for cls in (kvr.Kv4Layout, kvr.Kv8Layout, kvr.PagedLayout)]
    return {4: make[0](), 8: make[1](), 16: make[2]()}


def _calls(pool):
    """Every call that reads or writes a quantised pool, by the bits it is made for."""
    table, lin = _z(F32, 300, 32, 2), kvr.LinearLayout.empty(9, 2, device="cpu")
    k, v, q = _z(BF, 5, 2, 192), _z(BF, 5, 2, 128), _z(BF, 3, 16, 192)
    chunks = (_z(I32, 3), _z(I64, 2), _z(I32, 2))
    return [
        (4, lambda: kvr.kv4_append_rope(k, v, _z(I64, 5), _z(I32, 5), table, 0.7, pool)),
        (4, lambda: kvr.kv4_append_rope(k, v, _z(I64, 5), None, table, 0.7, pool, slots=_z(I64, 5))),
        (4, lambda: kvr.full_attn_decode_kv4(q, _z(I64, 3), _z(I32, 3), pool, table, 0.1, 100)),
        (4, lambda: kvr.kv4_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3), lin)),
        (8, lambda: kvr.kv8_append_rope(k, v, *chunks, table, 0.7, pool)),
        (8, lambda: kvr.full_attn_decode_kv8(q, _z(I64, 3), _z(I32, 3), pool, table, 0.1, 100)),
        (8, lambda: kvr.kv8_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 3), lin)),
    ]


@pytest.mark.parametrize("kind", [4, 8, 16])
def test_a_pool_of_other_bits_is_refused(rec, kind):  # noqa: F811
    for bits, call in _calls(_pools()[kind]):
        if bits == kind:
            call()
        else:
            n = len(rec.calls)
            with pytest.raises(TypeError):
                call()
            assert not [name for name, _ in rec.calls[n:] if not name.endswith("workspace_size")]


class _Pool4:
    """A caller's own 4-bit pool: the struct and its tensors, and no more."""

    def __init__(self):
        self.inner = kvr.Kv4Layout.contiguous(3, 2, 100, block_size=32, device="cpu")
        self.num_kv_heads = 2

    def tensors(self):
        return self.inner.tensors()

    def c(self):
        return self.inner.c()


def test_a_callers_own_4_bit_pool_is_taken(rec):  # noqa: F811
    for bits, call in _calls(_Pool4()):
        if bits == 4:
            call()
        else:
            with pytest.raises(TypeError):
                call()
    assert [n for n, _ in rec.calls if not n.endswith("workspace_size")] == ["kv4_append_rope", "kv4_append_rope",
                                                                            "full_attn_decode_kv4", "kv4_unpack"]


def test_the_first_wrong_argument_is_named(rec):  # noqa: F811
    """Of several wrong arguments the refusal names the one that comes first in the call's checks: queries, positions,
    lengths, the workspace, the output; entries ahead of the destination."""
    pool, table = _pools()[4], _z(F32, 300, 32, 2)
    q, pos, seq = _z(BF, 3, 16, 192), _z(I64, 3), _z(I32, 3)
    ws, odd = _z(torch.uint8, 8192), _z(BF, 3, 16, 192)
    for args, kw, name in (((q.float(), pos.int(), seq, pool, table), {}, "q must be"),
                           ((q, pos.int(), seq, None, table), {}, "pos must be"),
                           ((q, pos, _z(I32, 2), pool, table), dict(out=odd), "seq must have"),
                           ((q, pos, seq, pool, table), dict(workspace=ws.int(), out=odd), "workspace must be"),
                           ((q, pos, seq, pool, table), dict(workspace=ws, out=odd), "out must be")):
        with pytest.raises((TypeError, ValueError), match=name):
            kvr.full_attn_decode_kv4(*args, 0.1, 100, **kw)
    with pytest.raises(TypeError, match="lo must be"):
        kvr.kv4_unpack(pool, _z(I32, 2), _z(I32, 2), _z(I32, 3), None)
    with pytest.raises(ValueError, match="cu_rows must have"):
        kvr.kv4_unpack(pool, _z(I32, 2), _z(I64, 2), _z(I32, 2), None)


def test_cpu_tensors_are_refused_where_there_is_no_gpu():
    """With the library itself, and whether or not a GPU is there: the tensor that is not on one is named."""
    class Pool:
        data = block_table = None
        num_kv_heads = 2

        def __init__(self, tile):
            self.TILE = tile

    p4, p8 = Pool(kvr.KV4_TILE), Pool(kvr.KV8_TILE)
    table, k, v, q = _z(F32, 300, 32, 2), _z(BF, 5, 2, 192), _z(BF, 5, 2, 128), _z(BF, 3, 16, 192)
    bt, refs, ids, one, pairs, two = _z(I32, 3, 4), _z(I32, 12), _z(I32, 12), _z(I32, 1), _z(I32, 12), _z(I32, 2)
    for call, name in ((lambda: kvr.kv4_append_rope(k, v, _z(I64, 5), _z(I32, 5), table, 0.7, p4), "k"),
                       (lambda: kvr.full_attn_decode_kv4(q, _z(I64, 3), _z(I32, 3), p4, table, 0.1, 100), "q"),
                       (lambda: kvr.kv4_unpack(p4, two, _z(I64, 2), _z(I32, 3), None), "src_seqs"),
                       (lambda: kvr.kv8_append_rope(k, v, _z(I32, 3), _z(I64, 2), two, table, 0.7, p8), "k"),
                       (lambda: kvr.full_attn_decode_kv8(q, _z(I64, 3), _z(I32, 3), p8, table, 0.1, 100), "q"),
                       (lambda: kvr.kv8_unpack(p8, two, _z(I64, 2), _z(I32, 3), None), "src_seqs"),
                       (lambda: kvr.kv_pages_free(bt, 12, 32, refs, two, ids, one), "block_table"),
                       (lambda: kvr.kv_pages_fork(bt, 12, 32, refs, two, two, _z(I64, 2), ids, one, pairs, pairs, one), "block_table"),
                       (lambda: kvr.kv_pages_compact(bt, 12, refs, ids, one, pairs, pairs, one), "block_table")):
        with pytest.raises(ValueError, match=f"^{name} must be a CUDA tensor"):
            call()
