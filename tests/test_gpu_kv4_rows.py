"""kv4_unpack of entries whose cu_rows is out of order or runs past the rows: the call
says so, and up to 64 entries those ahead of the place are written."""
import numpy as np
import pytest
import torch

import sinks_kv_ring_gb300 as kvr

from test_gpu_kv4_unpack import DEV, _built, _filled, _ints, _want, table  # noqa: F401
from test_gpu_kv8_rows import ORDERS, _served

pytestmark = pytest.mark.gpu


def _check(src, seqs, cu, T, hkv, flags, served, first):
    n = len(cu) - 1
    out = kvr.LinearLayout(torch.full((T, hkv, 192), 7.0, dtype=torch.bfloat16, device=DEV),
                           torch.full((T, hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV))
    kvr.kv4_unpack(src, _ints(seqs, torch.int32), _ints([first] * n, torch.int64), _ints(cu, torch.int32), out)
    said = kvr.device_status()
    assert said & flags if served < n else said == flags
    behind = torch.zeros(T, dtype=torch.bool, device=DEV)
    for a, b in zip(cu[served:], cu[served + 1:]):
        behind[max(a, 0):max(b, 0)] = True
    for i in range(served):
        if cu[i] < cu[i + 1]:
            keep = ~behind[cu[i]:cu[i + 1]]
            for got, want in zip((out.k, out.v), _want(src, seqs[i], first, cu[i + 1] - cu[i])):
                assert torch.equal(got[cu[i]:cu[i + 1]][keep], want[keep]), i


@pytest.mark.parametrize("name", list(ORDERS))
def test_out_of_order(table, name):  # noqa: F811
    cu, T = ORDERS[name]
    n, hkv, gen = len(cu) - 1, 2, torch.Generator(device=DEV).manual_seed(len(name))
    src = _filled(gen, 3, hkv, 128, 32, table)
    good = _served(cu, T)
    _check(src, [i % 3 for i in range(n)], cu, T, hkv, kvr.DEV_BAD_ROWS, good, 5)


@pytest.mark.parametrize("n", [3, 33, 64])
@pytest.mark.parametrize("mean", [1, 12])
def test_one_place_out_of_order(table, mean, n):  # noqa: F811
    rng, gen = np.random.default_rng(n + mean), torch.Generator(device=DEV).manual_seed(n)
    src = _filled(gen, 3, 3, 2 * mean * n + 16, 16, table)
    for case in range(5):
        cu = np.concatenate([[0], np.cumsum(rng.integers(0, 2 * mean + 1, n))]).astype(np.int64)
        T = max(int(cu[-1]), 1)
        at = int(rng.integers(0, n + 1))
        if case < 4:
            cu[at] = (-1 - int(rng.integers(0, 1000)), T + 1, int(rng.integers(0, T + 1)), 0)[case]
        cu = cu.tolist()
        good = _served(cu, T)
        _check(src, rng.integers(0, 3, n).tolist(), cu, T, 3, kvr.DEV_BAD_ROWS if good < n else 0, good, 3)


@pytest.mark.parametrize("n", [65, 5000])
def test_out_of_order_among_many(table, n):  # noqa: F811
    gen = torch.Generator(device=DEV).manual_seed(n)
    src = _filled(gen, 1, 1, 16, 16, table)
    for at, to in ((n // 2, 7), (n, n + 1), (n - 1, -1), (0, -1)):
        cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
        cu[at] = to
        kvr.kv4_unpack(src, torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV), cu,
                       kvr.LinearLayout.empty(n, 1))
        assert kvr.device_status() & kvr.DEV_BAD_ROWS
