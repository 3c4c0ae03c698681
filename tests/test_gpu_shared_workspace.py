"""GPU test that decode_shared stays within the workspace that it asks for, with states of many ragged groups beside each
other.  Tolerances as test_gpu_shared."""
import numpy as np
import pytest
import torch

from _gpu_support import f64
from _shared_support import SharedCache
from test_gpu_shared import _check, _q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 64, 8, 128), ("bf16", 32, 32, 64), ("bf16", 8, 8, 128), ("fp8", 64, 8, 128)])
@pytest.mark.parametrize("groups", [
    [(512, [513 + i % 7 for i in range(n)]) for n in (2, 3, 1, 33, 0, 2, 65, 5)],
    [(160 + 16 * (i % 5), [300] * 2) for i in range(60)],
    [(600, [601 + i % 50 for i in range(100)])],
])
def test_stays_within(kvattn_lib, dtype, hq, hkv, d, groups):
    kv = kvattn_lib
    groups = [g for g in groups if g[1]]
    c = SharedCache(kv, dtype, hkv, d, groups, seed=len(groups))
    cfg = kv.make_config(hq, hkv, d, kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    q = _q(np.random.default_rng(hq), (len(c.lens), hq, d), dtype)
    for most in (int(c.shared.max()), 1 << 16):
        size = kv.decode_shared_workspace_size(cfg, len(c.lens), max(c.lens), len(c.shared), most)
        space = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q, device="cuda")
        call(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, max(c.lens), c.d_cu, c.d_shared, most, out=out,
             workspace=space[:size])
        assert kv.get_device_status() == 0
        assert bool((space[size:] == 0xA5).all())
        _check(c, q, f64(out), dtype, f"bound {most}")
