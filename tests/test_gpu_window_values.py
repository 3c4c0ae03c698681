"""GPU tests of the windowed attentions on values at the ends of their ranges, against the formula in 64 bits: NaN that
a query sees, V scales far apart, calls that are refused, long sequences."""
import numpy as np
import pytest
import torch

from _window_support import TORCH_DT, WindowCache, attend, check_attention, seen
from _gpu_support import f64

pytestmark = pytest.mark.gpu


def _q(seed, shape, dtype="bf16"):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).to(TORCH_DT["f32" if dtype == "f32" else "bf16"])


def _at(c, r, token):
    """Block id and slot of a token of sequence r."""
    block = c.cache.block_size
    return int(c.table[r, token // block]), token % block


def _nan_key(c, r, token, head):
    b, s = _at(c, r, token)
    if c.dtype == "fp8":  # its scale
        c.cache.pool[b, head, s // 16, 4096 + 4 * (s % 16):4100 + 4 * (s % 16)] = torch.tensor(
            [float("nan")], device="cuda").view(torch.uint8)
    else:
        c.cache.k_pool[b, head, s] = float("nan")
    c.k[r][token, head] = float("nan")


def _check_with_nan(got, want, mag, dtype, what):
    """NaN where the formula has NaN and only there; the other heads within the bound."""
    bad = np.isnan(want).all(-1)
    assert np.array_equal(np.isnan(want).any(-1), bad)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN lost or made"
    check_attention(got[~bad][:, None], want[~bad][:, None], mag[~bad][:, None], dtype, what)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 8, 2, 64), ("bf16", 2, 2, 128), ("fp8", 8, 2, 128),
                                            ("f32", 8, 2, 128), ("f32", 4, 4, 64)])
@pytest.mark.parametrize("splits", [0, 3])
def test_decode_seen_nan(kvattn_lib, dtype, hq, hkv, d, splits):
    """NaN in a query row, and in a key that is seen (the only one of its tile at 17, 33 and 4001 keys): the softmax of
    that head is NaN however its tiles are shared out."""
    kv = kvattn_lib
    lens, window, sinks = [17, 33, 40, 5, 4001, 600], 3000, 3
    wanted = [seen([L - 1], L, window, sinks)[0] for L in lens]
    c = WindowCache(kv, dtype, hkv, d, lens, wanted, seed=2)
    q = _q(3, (len(lens), hq, d), dtype)
    q[5, 1, 7] = float("nan")                       # one element of one query head
    for r, token in ((0, 16), (1, 32), (2, 39), (4, 4000), (4, 1500)):
        _nan_key(c, r, token, (token % 2) % hkv)
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_window_fp8 if dtype == "fp8" else kv.decode_window
    out = call(cfg, c.cache, q.cuda(), c.d_table, torch.tensor(lens, dtype=torch.int32).cuda(), max(lens), window, sinks,
               num_splits=splits)
    assert kv.get_device_status() == 0
    got = f64(out)
    for r, L in enumerate(lens):
        want, mag = attend(q[r:r + 1].double().numpy(), c.k[r], c.v[r], wanted[r][None])
        _check_with_nan(got[r:r + 1], want, mag, dtype, f"length {L}")
    assert np.isnan(got[0]).any() and np.isnan(got[5, 1]).all()


def test_one_row_with_nan_is_the_same_in_both(kvattn_lib):
    """A chunk of one row and a single token: NaN in the same heads."""
    kv = kvattn_lib
    lens = [17, 300]
    wanted = [seen([L - 1], L, 100, 4)[0] for L in lens]
    for dtype in ("bf16", "fp8"):
        c = WindowCache(kv, dtype, 2, 128, lens, wanted, seed=4)
        q = _q(5, (2, 8, 128)).cuda()
        q[1, 6, 0] = float("nan")
        _nan_key(c, 0, 16, 0)
        cfg = kv.make_config(8, 2, 128, kv.BF16)
        n = torch.tensor(lens, dtype=torch.int32).cuda()
        dec, pre = (kv.decode_window_fp8, kv.prefill_window_fp8) if dtype == "fp8" else (kv.decode_window, kv.prefill_window)
        a = dec(cfg, c.cache, q, c.d_table, n, 300, 100, 4)
        b = pre(cfg, c.cache, q, torch.arange(3, dtype=torch.int32).cuda(), n - 1, c.d_table, 1, 100, 4)
        assert kv.get_device_status() == 0
        heads = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
        heads[0, :4] = heads[1, 6] = True
        for got in (a, b):
            assert torch.equal(torch.isnan(got).all(-1), heads) and torch.equal(torch.isnan(got).any(-1), heads)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_decode_of_the_whole_cache_seen_nan(kvattn_lib, dtype, splits):
    """The same of kvattn_decode, whose kernels the windowed form shares."""
    kv = kvattn_lib
    lens = [17, 33, 2001, 600]
    wanted = [np.ones(L, bool) for L in lens]
    c = WindowCache(kv, dtype, 2, 128, lens, wanted, seed=2)
    q = _q(3, (len(lens), 8, 128), dtype)
    q[3, 1, 7] = float("nan")
    for r, token in ((0, 16), (1, 32), (2, 2000)):
        _nan_key(c, r, token, r % 2)
    cfg = kv.make_config(8, 2, 128, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_fp8 if dtype == "fp8" else kv.decode
    out = call(cfg, c.cache, q.cuda(), c.d_table, torch.tensor(lens, dtype=torch.int32).cuda(), max(lens), num_splits=splits)
    assert kv.get_device_status() == 0
    got = f64(out)
    for r, L in enumerate(lens):
        want, mag = attend(q[r:r + 1].double().numpy(), c.k[r], c.v[r], wanted[r][None])
        _check_with_nan(got[r:r + 1], want, mag, dtype, f"length {L}")
