"""GPU tests of compaction lists that count as empty: their sequences stay as they were, the others move."""
import numpy as np
import pytest
import torch

from test_gpu_compact import KINDS, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,layers", KINDS)
@pytest.mark.parametrize("start", [-1, -2 ** 31, 108, 2 ** 31 - 3])
def test_lists_without_places(kvattn_lib, dtype, layers, start):
    """A negative first place, or five tokens from a place on that leaves fewer in the table's 112."""
    kv = kvattn_lib
    lists = [[3, 5, 50, 99], [12, 30, 31, 32, 90], [1, 2, 64]]
    c = Case(kv, dtype, layers, 2, 128, [100, 100, 100], [0, 10, 0], lists, seed=8)
    c.ints[1][1] = start
    c.run()
    assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    c.lists[1] = []
    assert np.array_equal(c.raw.cpu().numpy(), c.want())


@pytest.mark.parametrize("dtype,layers", KINDS)
def test_one_long_list_among_many(kvattn_lib, dtype, layers):
    """A list far longer than the mean one, the others empty or of a few tokens."""
    g = np.random.default_rng(9)
    lens = [6000] + [20] * 40 + [1] * 20
    lists = [[p for p in range(6000) if g.random() < 0.5]] + [[p for p in range(20) if g.random() < 0.5] for _ in range(40)]
    c = Case(kvattn_lib, dtype, layers, 3, 128, lens, [0] * len(lens), lists + [[]] * 20, seed=9)
    c.run()
    c.check()
