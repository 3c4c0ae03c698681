"""GPU tests of shared decode over prefixes of which blocks are missing from the table: their tokens are seen by nobody, in
either form of the call, whatever the shared memory of the GPU held before.  Tolerances as test_gpu_shared."""
import numpy as np
import pytest
import torch

from _gpu_support import f64
from _shared_support import SharedCache
from _window_support import WindowCache, attend, check_attention
from test_gpu_shared import LOOSE, _q

pytestmark = pytest.mark.gpu


def _nan_everywhere(kv, cfg, call, c, q):
    """A call over a cache of NaN only: tiles of it stay in the shared memory of every SM."""
    if hasattr(c.cache, "pool"):
        nan = kv.CacheFP8(torch.full_like(c.cache.pool, 0xFF), c.cache.block_size)
    else:
        nan = kv.Cache(*(torch.full_like(p, float("nan")) for p in (c.cache.k_pool, c.cache.v_pool)))
    call(cfg, nan, q, c.d_table, c.d_lens, max(c.lens), c.d_cu, c.d_shared, LOOSE)


def _check(c, q, got, dtype, gone, rows, what):
    """`gone`: the tokens that are missing of each of `rows`."""
    for r in rows:
        n = c.lens[r]
        seen = np.ones((1, n), bool)
        seen[0, [t for t in gone(r) if t < n]] = False
        want, mag = attend(q[r:r + 1], c.k[r], c.v[r], seen)
        check_attention(got[r:r + 1], want, mag, "f32" if dtype == "f32" else "bf16", f"{what}, sequence {r}")


HEADS = [("bf16", 32, 8, 128, 4), ("bf16", 12, 12, 64, 4), ("bf16", 64, 8, 128, 40), ("fp8", 64, 8, 128, 4),
         ("fp8", 32, 8, 128, 40), ("f32", 8, 2, 128, 4)]


@pytest.mark.parametrize("dtype,hq,hkv,d,n", HEADS)
@pytest.mark.parametrize("gone", [[0], [20], [3, 4, 5, 37], [8, 9, 10, 11, 12, 13, 14, 15], list(range(43))])
def test_missing_of_all(kvattn_lib, dtype, hq, hkv, d, n, gone):
    """The same blocks are missing from every row of a group: one, some of a tile, a whole tile, the whole prefix."""
    kv = kvattn_lib
    c = SharedCache(kv, dtype, hkv, d, [(700, [701 + 13 * i % 64 for i in range(n)]), (0, [40])], seed=len(gone))
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    q = _q(np.random.default_rng(gone[0]), (n + 1, hq, d), dtype)
    tokens = [16 * b + t for b in gone for t in range(16)]
    for block in (-1, c.cache.num_blocks, 2 ** 31 - 1):
        table = c.d_table.clone()
        table[:n, gone] = block
        for most in (700, LOOSE):
            _nan_everywhere(kv, cfg, call, c, q.cuda())
            kv.get_device_status()
            got = f64(call(cfg, c.cache, q.cuda(), table, c.d_lens, max(c.lens), c.d_cu, c.d_shared, most))
            assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
            _check(c, q.double().numpy(), got, dtype, lambda r: tokens if r < n else [], range(0, n + 1, max(1, n // 4)),
                   f"block {block}, bound {most}")


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 12, 12, 64), ("fp8", 32, 8, 128)])
def test_missing_of_one(kvattn_lib, dtype, hq, hkv, d):
    """Blocks that only one row lacks: the group lacks them where the prefix is read through that row, other groups and the
    sequences that do not have the whole prefix keep theirs."""
    kv = kvattn_lib
    groups = [(512, [530, 513, 600, 40]), (300, [301, 350])]
    c = SharedCache(kv, dtype, hkv, d, groups, seed=3)
    cfg = kv.make_config(hq, hkv, d, kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    q = _q(np.random.default_rng(4), (6, hq, d), dtype)
    table = c.d_table.clone()
    table[0, 5] = -1
    for most in (512, LOOSE):
        _nan_everywhere(kv, cfg, call, c, q.cuda())
        kv.get_device_status()
        got = f64(call(cfg, c.cache, q.cuda(), table, c.d_lens, max(c.lens), c.d_cu, c.d_shared, most))
        assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
        lacks = {0} if most == 512 else {0, 1, 2}  # (row 0 is the first that has them all)
        _check(c, q.double().numpy(), got, dtype, lambda r: range(80, 96) if r in lacks else [], range(6), f"bound {most}")


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 64, 8, 128), ("bf16", 8, 8, 128),
                                            ("bf16", 16, 8, 128), ("fp8", 64, 8, 128), ("fp8", 32, 8, 128),
                                            ("f32", 16, 8, 128), ("f32", 64, 8, 64)])
def test_missing_under_long_bounds(kvattn_lib, dtype, hq, hkv, d):
    """Calls that go to the balanced stream by their bound: a block that is not in the pool is seen by nobody there either,
    in decode_shared without groups and in decode_window."""
    kv = kvattn_lib
    c = SharedCache(kv, dtype, hkv, d, [(0, [701, 760, 33, 640, 16])], seed=5)
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    window = kv.decode_window_fp8 if dtype == "fp8" else kv.decode_window
    q = _q(np.random.default_rng(6), (5, hq, d), dtype)
    bound, none = 16 * 4200, torch.zeros(0, dtype=torch.int32, device="cuda")  # 5 * 8 * 4200 tiles: 65536 and more
    gone = {0: [0, 7, 43], 1: [20, 21, 22, 23, 47], 4: [0]}
    for block in (-1, c.cache.num_blocks):
        table = c.d_table.clone()
        for r, cols in gone.items():
            table[r, cols] = block
        # (block 0 is another sequence's: its keys must not stand in for the missing ones)
        got = f64(call(cfg, c.cache, q.cuda(), table, c.d_lens, bound, torch.zeros(1, dtype=torch.int32, device="cuda"), none,
                       0))
        assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
        lacks = lambda r: [16 * b + t for b in gone.get(r, []) for t in range(16)]  # noqa: E731
        _check(c, q.double().numpy(), got, dtype, lacks, range(4), f"block {block}")
        assert np.all(got[4] == 0)
        got = f64(window(cfg, c.cache, q.cuda(), table, c.d_lens, bound, bound - 5))
        assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
        _check(c, q.double().numpy(), got, dtype, lacks, range(4), f"window, block {block}")
        assert np.all(got[4] == 0)


@pytest.mark.parametrize("hq,hkv", [(64, 8), (32, 8)])
@pytest.mark.parametrize("scale", [-1.0, 0.0, -3.0e38])
def test_scales_of_unseen_slots(kvattn_lib, hq, hkv, scale):
    """Whatever the scales of slots are that the window does not see, in pages of which it sees others: the balanced stream
    over fp8 pages, which marks missing pages by scales of its own."""
    kv = kvattn_lib
    lens, window = [701, 760, 33, 640], 300
    wanted = [np.arange(n) >= n - window for n in lens]
    c = WindowCache(kv, "fp8", hkv, 128, lens, wanted, seed=hq)
    scales = c.cache.pool.view(torch.float32)[..., 1024:]  # K's and V's
    scales[torch.isnan(scales)] = scale
    cfg = kv.make_config(hq, hkv, 128, kv.BF16)
    q = _q(np.random.default_rng(7), (4, hq, 128), "fp8")
    d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = f64(kv.decode_window_fp8(cfg, c.cache, q.cuda(), c.d_table, d_lens, 16 * 4200, window))
    split = f64(kv.decode_window_fp8(cfg, c.cache, q.cuda(), c.d_table, d_lens, 16 * 4200, window, num_splits=3))
    assert kv.get_device_status() == 0
    for r in range(4):
        want, mag = attend(q[r:r + 1].double().numpy(), c.k[r], c.v[r], wanted[r][None])
        for x in (got, split):
            check_attention(x[r:r + 1], want, mag, "bf16", f"sequence {r}")
