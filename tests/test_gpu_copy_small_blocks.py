"""GPU tests of block copies whose runs are far smaller than what a thread block moves at a time."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 2, 37, 700, 3001])
@pytest.mark.parametrize("dtype,hkv,d,block,layers", [
    ("bf16", 1, 64, 16, 5), ("bf16", 1, 64, 16, 1), ("bf16", 1, 64, 1, 3), ("bf16", 1, 128, 3, 2), ("bf16", 3, 64, 16, 2),
    ("bf16", 2, 128, 16, 1), ("bf16", 9, 64, 16, 2), ("f32", 1, 64, 16, 2), ("f32", 5, 64, 5, 1), ("fp8", 1, 128, 16, 1),
    ("fp8", 3, 128, 16, 1), ("fp8", 1, 128, 32, 1)])
def test_copies(kvattn_lib, dtype, hkv, d, block, layers, n):
    """Every pair's blocks, nothing else; pairs with a bad id are skipped and reported."""
    kv = kvattn_lib
    g = np.random.default_rng(n + hkv)
    blocks = 2 * n + 5
    cfg = kv.make_config(hkv, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    if dtype == "fp8":
        pool = torch.randint(0, 256, (blocks, hkv, block // 16, 4224), dtype=torch.uint8, device="cuda")
        cache, regions = kv.CacheFP8(pool, block), [pool]
    elif layers == 1:
        regions = [torch.randn((blocks, hkv, block, d), device="cuda").to(torch.float32 if dtype == "f32" else torch.bfloat16)
                   for _ in range(2)]
        cache = kv.Cache(*regions)
    else:
        pool = torch.randn((layers, 2, blocks, hkv, block, d), device="cuda")
        pool = pool.to(torch.float32 if dtype == "f32" else torch.bfloat16)
        cache, regions = kv.LayeredCache(cfg, pool), list(pool.flatten(0, 1))
    ids = g.permutation(blocks)
    src, dst = ids[:n].astype(np.int32), ids[n:2 * n].astype(np.int32)
    for wrong in (False, True):
        good = np.ones(n, bool)
        if wrong:
            bad = g.choice(n, max(1, n // 7), replace=False)
            good[bad] = False
            for i, b in enumerate(bad):
                (src if i % 2 else dst)[b] = (-1, blocks, 2 ** 31 - 1)[i % 3]
        want = [r.clone() for r in regions]
        for w in want:
            w[torch.from_numpy(dst[good].astype(np.int64)).cuda()] = w[torch.from_numpy(src[good].astype(np.int64)).cuda()]
        kv.copy_blocks(cfg, cache, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
        assert kv.get_device_status() == (kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"] if wrong else 0)
        for r, w in zip(regions, want):
            assert torch.equal(r.view(torch.uint8), w.view(torch.uint8))
