"""GPU test of block copies on a stream that is not the current one, the ids given as lists."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["rows", "layers", "fp8"])
def test_ids_outlive_the_call(kvattn_lib, kind):
    """The uploaded ids stay what they are until the copy, which is behind other work of its stream, has read them: memory
    that the current stream is given meanwhile is not theirs."""
    kv = kvattn_lib
    hkv, d, blocks, n = 2, 128, 64, 16
    cfg = kv.make_config(8, hkv, d, kv.BF16)
    if kind == "fp8":
        pool = torch.randint(0, 100, (blocks, hkv, 1, 4224), dtype=torch.uint8, device="cuda")
        cache, pools = kv.CacheFP8(pool), [pool]
    elif kind == "layers":
        pool = torch.randn((3, 2, blocks, hkv, 16, d), device="cuda").bfloat16()
        cache, pools = kv.LayeredCache(cfg, pool), [p for p in pool.flatten(0, 1)]
    else:
        pools = [torch.randn((blocks, hkv, 16, d), device="cuda").bfloat16() for _ in range(2)]
        cache = kv.Cache(*pools)
    src, dst = list(range(n)), list(range(32, 32 + n))
    want = [p.clone() for p in pools]
    for w in want:
        w[dst] = w[src]
    side = torch.cuda.Stream()
    for _ in range(3):  # (the allocator holds memory of this size already, and every kernel is loaded, as in a running server)
        kv.copy_blocks(cfg, cache, src, src)
        torch.full((n,), 63, dtype=torch.int32, device="cuda")
        torch.cuda._sleep(100)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    kv.copy_blocks(cfg, cache, src, dst, stream=side)
    others = [torch.full((n,), 63, dtype=torch.int32, device="cuda") for _ in range(64)]  # valid ids, of other blocks
    torch.cuda.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    assert len(others) == 64 and kv.get_device_status() == 0
