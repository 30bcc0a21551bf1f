"""kv_pages_compact over free lists and counts that are none: nothing moves, and arrays
apart from the inputs receive the inputs."""
import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr
from oracle import pages_share as ops

from test_gpu_pages_share import DEV, _built, _t  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nb,cap", [(1, 1), (10, 10), (10, 30), (40, 7), (3000, 20000), (20000, 20000)])
def test_compact_leaves_what_it_cannot_read(nb, cap):
    rng = np.random.default_rng(nb + cap)
    S, mb = 5, 9
    table = rng.integers(-1, nb, (S, mb)).astype(np.int32)
    refs = rng.integers(0, 3, nb).astype(np.int32)
    lists = [np.arange(cap) % nb, np.arange(cap) + 1, np.full(cap, -1)]      # names repeat, run past the pool, are none
    for free in lists:
        for count in (-1, -(1 << 31), 1, cap // 2, cap, cap + 1, nb, nb + 1, (1 << 31) - 1):
            wt, wr, wf, pairs, flags = ops.compact(table, refs, free, count)
            if flags == 0:
                continue
            t, r, f, c = _t(table), _t(refs), _t(free), _t([count])
            out = [torch.full_like(x, 77) for x in (t, r, f)]
            a, b, k = _t([5] * max(nb // 2, 1)), _t([5] * max(nb // 2, 1)), _t([5])
            kvr.kv_pages_compact(t, nb, r, f, c, a, b, k, table_out=out[0], refs_out=out[1], free_ids_out=out[2])
            assert kvr.device_status() == flags and int(k) == 0
            n = min(max(count, 0), cap)
            assert torch.equal(out[0], t) and torch.equal(out[1], r), (count, free[:3])
            assert torch.equal(out[2][:n], f[:n]) and (out[2][n:] == 77).all(), (count, free[:3])
            assert np.array_equal(t.cpu().numpy(), table) and int(c) == count
