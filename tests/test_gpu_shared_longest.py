"""GPU test of decode_shared at the longest lengths that an int32 holds, over tables that name the same few blocks again
and again."""
import numpy as np
import pytest
import torch

from _gpu_support import f64
from _shared_support import SharedCache
from _window_support import attend
from test_gpu_shared import LOOSE, _check, _q

pytestmark = pytest.mark.gpu


def test_longest(kvattn_lib):
    """Lengths of which a count of pages rounded up passes 2^31.  A repeated list of keys weighs as once, so the result is
    the softmax over the 64 blocks (a last part of a round of them, below 2^-20 of the whole, aside).  A warp adds at most
    2^28 / 1200 = 2.3e5 pages to its sums one by one: each fp32 addition is off by at most 2^-24 of the sum (P.V on the
    tensor cores, which may cut: 2^-23), together less than 2^-6 and 2^-5; the weights' rounding is 2^-8."""
    kv = kvattn_lib
    hq, hkv, d, blocks, width = 8, 1, 64, 64, 1 << 27
    g = np.random.default_rng(1)
    pools = [torch.from_numpy(g.standard_normal((blocks, hkv, 16, d))).to(torch.bfloat16) for _ in range(2)]
    cache = kv.Cache(*(p.cuda() for p in pools))
    table = (torch.arange(width, dtype=torch.int32, device="cuda") % blocks).repeat(2, 1)
    lens = [2 ** 31 - 1, 2 ** 31 - 14]
    q = _q(g, (2, hq, d), "bf16")
    cfg = kv.make_config(hq, hkv, d, kv.BF16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    got = f64(kv.decode_shared(cfg, cache, q.cuda(), table, i32(*lens), 2 ** 31 - 1, i32(0, 2), i32(1 << 20), 1 << 20))
    assert kv.get_device_status() == 0
    k, v = (f64(p).swapaxes(1, 2).reshape(-1, hkv, d) for p in pools)
    for r in range(2):
        want, mag = attend(q[r:r + 1].double().numpy(), k, v, np.ones((1, len(k)), bool))
        assert np.all(np.abs(got[r] - want[0]) <= (2.0 ** -6 + 2.0 ** -5 + 2.0 ** -7) * mag[0])


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 4, 4, 64), ("fp8", 32, 8, 128), ("f32", 8, 2, 64)])
def test_bound_of_any_length(kvattn_lib, dtype, hq, hkv, d):
    """max_seq_len 2^31 - 1, "no bound", over short sequences: in decode_shared and decode_window."""
    kv = kvattn_lib
    c = SharedCache(kv, dtype, hkv, d, [(300, [301, 340, 17]), (0, [40])], seed=2)
    q = _q(np.random.default_rng(3), (4, hq, d), dtype)
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    fp8 = dtype == "fp8"
    for most in (300, LOOSE):
        got = (kv.decode_shared_fp8 if fp8 else kv.decode_shared)(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, 2 ** 31 - 1,
                                                                  c.d_cu, c.d_shared, most)
        assert kv.get_device_status() == 0
        _check(c, q, f64(got), dtype, f"bound {most}")
    got = (kv.decode_window_fp8 if fp8 else kv.decode_window)(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, 2 ** 31 - 1,
                                                              2 ** 31 - 1)
    assert kv.get_device_status() == 0
    _check(c, q, f64(got), dtype, "window")
