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
