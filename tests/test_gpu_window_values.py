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


def _v_size(c, r, times, zero=()):
    """Multiplies the V rows of sequence r of an fp8 cache by times[token] (powers of two: exact), and makes the rows
    `zero` zeros as they are stored: codes of 0 and the scale 1."""
    pool = c.cache.pool
    for token in np.nonzero(c.table[r, np.arange(len(times)) // c.cache.block_size] >= 0)[0]:
        b, s = _at(c, r, int(token))
        page = pool[b, :, s // 16]
        at = 4160 + 4 * (s % 16)
        scale = page[:, at:at + 4].contiguous().view(torch.float32)
        if token in zero:
            page[:, 2048 + s % 16:4096:16] = 0
            scale = torch.ones_like(scale)
        else:
            scale = scale * float(times[token])
        page[:, at:at + 4] = scale.view(torch.uint8)
    c.v[r] = c.v[r] * np.asarray(times)[:, None, None]
    c.v[r][list(zero)] = 0.0


@pytest.mark.parametrize("case", ["zero rows", "no weight", "by token", "tiny"])
@pytest.mark.parametrize("splits", [0, 3])
def test_decode_fp8_v_of_any_size(kvattn_lib, case, splits):
    """V rows of very different sizes: rows of zeros (stored with the scale 1) among small ones, a row 2^30 times the
    others whose weight is 2^-150, sizes from 1 to 2^-23 by token, all of 2^-90."""
    kv = kvattn_lib
    lens, window, sinks, hkv, g = [1024, 17, 300, 1], 800, 2, 2, 4
    wanted = [seen([L - 1], L, window, sinks)[0] for L in lens]
    c = WindowCache(kv, "fp8", hkv, 128, lens, wanted, seed=6)
    q = _q(7, (len(lens), hkv, 1, 128)).expand(len(lens), hkv, g, 128).reshape(len(lens), hkv * g, 128).contiguous()
    for r, L in enumerate(lens):
        t, zero = np.ones(L), ()
        if case == "zero rows":
            t *= 2.0 ** -20
            zero = sorted({0, L - 1, max(0, L - 6)})
        elif case == "by token":
            t = 2.0 ** -(np.arange(L) % 24).astype(np.float64)
        elif case == "tiny":
            t *= 2.0 ** -90
        elif L > 100:  # the key of the lowest score of each head, which 2^6 times as long weighs under 2^-150
            for h in range(hkv):
                s = np.where(wanted[r], c.k[r][:, h] @ q[r, h * g].double().numpy() / np.sqrt(128.0), 0.0)
                low = int(s.argmin())
                assert s[low] * 2.0 ** 6 < -150 * np.log(2.0)
                b, at = _at(c, r, low)
                page = c.cache.pool[b, h, at // 16]
                for off, times in ((4096, 2.0 ** 6), (4160, 2.0 ** 30)):
                    w = page[off + 4 * (at % 16):off + 4 * (at % 16) + 4]
                    w.copy_((w.clone().view(torch.float32) * times).view(torch.uint8))
                c.k[r][low, h] *= 2.0 ** 6
                c.v[r][low, h] *= 2.0 ** 30
        _v_size(c, r, t, zero)
    out = kv.decode_window_fp8(kv.make_config(hkv * g, hkv, 128, kv.BF16), c.cache, q.cuda(), c.d_table,
                               torch.tensor(lens, dtype=torch.int32).cuda(), max(lens), window, sinks, num_splits=splits)
    assert kv.get_device_status() == 0
    for r, L in enumerate(lens):
        want, mag = attend(q[r:r + 1].double().numpy(), c.k[r], c.v[r], wanted[r][None])
        # the roundings of check_attention; a product of a weight and a V scale loses at most 2^-25 of the largest
        # besides, and of 800 keys those together are far below the 2^-10 of sum w |v| that the bound has to spare
        check_attention(f64(out)[r:r + 1], want, mag, "fp8", f"{case}, length {L}")


@pytest.mark.parametrize("size", [2.0 ** -30, 1.0, 2.0 ** 30])
def test_prefill_fp8_rows_of_zeros(kvattn_lib, size):
    """V rows of zeros, stored with the scale 1, among rows far smaller and larger than 1; K rows of zeros too."""
    kv = kvattn_lib
    chunks, window, sinks, zero = [(100, 200), (0, 70)], 120, 4, [0, 3, 40, 60, 101, 299]
    masks = [seen(range(p, p + n), p + n, window, sinks) for p, n in chunks]
    c = WindowCache(kv, "fp8", 2, 128, [300, 70], [m.any(0) for m in masks], seed=3)
    for r, m in enumerate(masks):
        mine = [t for t in zero if t < m.shape[1]]
        _v_size(c, r, np.full(m.shape[1], size), mine)
        for token in mine:
            if m.any(0)[token]:
                b, s = _at(c, r, token)
                c.cache.pool[b, :, s // 16, 128 * (s % 16):128 * (s % 16) + 128] = 0
                c.cache.pool[b, :, s // 16, 4096 + 4 * (s % 16):4100 + 4 * (s % 16)] = torch.ones(1).view(torch.uint8).cuda()
                c.k[r][token] = 0.0
    q = _q(1, (270, 8, 128))
    out = kv.prefill_window_fp8(kv.make_config(8, 2, 128, kv.BF16), c.cache, q.cuda(),
                                torch.tensor([0, 200, 270], dtype=torch.int32).cuda(),
                                torch.tensor([100, 0], dtype=torch.int32).cuda(), c.d_table, 200, window, sinks)
    assert kv.get_device_status() == 0
    for i, (a, b) in enumerate([(0, 200), (200, 270)]):
        want, mag = attend(q[a:b].double().numpy(), c.k[i], c.v[i], masks[i])
        check_attention(f64(out)[a:b], want, mag, "fp8", f"chunk {i}")


def test_prefill_fp8_infinite_key_of_a_later_row(kvattn_lib):
    """An infinite key (its scale) that only the chunk's last row sees: the other rows keep the precision of their small
    keys."""
    kv = kvattn_lib
    n, window, sinks, small = 150, 60, 2, 2.0 ** -17
    mask = seen(range(n), n, window, sinks)
    c = WindowCache(kv, "fp8", 2, 128, [n], [mask.any(0)], seed=9)
    ks = c.cache.pool[..., 4096:4160].contiguous().view(torch.float32) * small
    b, s = _at(c, 0, n - 1)
    ks[b, :, s // 16, s % 16] = float("inf")
    c.cache.pool[..., 4096:4160] = ks.view(torch.uint8)
    q = _q(2, (n, 8, 128)) / small
    out = kv.prefill_window_fp8(kv.make_config(8, 2, 128, kv.BF16), c.cache, q.cuda(),
                                torch.tensor([0, n], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                                c.d_table, n, window, sinks)
    assert kv.get_device_status() == 0
    want, mag = attend(q[:-1].double().numpy(), c.k[0] * small, c.v[0], mask[:-1])
    check_attention(f64(out)[:-1], want, mag, "fp8", "rows before")


def test_prefill_fp8_refusal_launches_nothing(kvattn_lib):
    """More work items than can be numbered, by a max_q_len far past the chunk's: refused before the workspace is
    touched, in the plain form as well."""
    kv = kvattn_lib
    hq, hkv, n, window, sinks, most = 128, 32, 20, 16, 2, 2 ** 31 - 1
    c = WindowCache(kv, "fp8", hkv, 128, [n], [np.ones(n, bool)], seed=1)
    cfg = kv.make_config(hq, hkv, 128, kv.BF16)
    q = _q(2, (n, hq, 128)).cuda()
    cu, prefix = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    ws = torch.full((kv.prefill_window_fp8_workspace_size(cfg, 16, c.d_table.shape[1], 1, most, window, sinks),), 77,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 9.0)
    with pytest.raises(kv.KvattnError, match="UNSUPPORTED"):
        kv.prefill_window_fp8(cfg, c.cache, q, cu, prefix, c.d_table, most, window, sinks, out=out, workspace=ws)
    c16 = WindowCache(kv, "bf16", hkv, 128, [n], [np.ones(n, bool)], seed=1)
    with pytest.raises(kv.KvattnError, match="UNSUPPORTED"):
        kv.prefill_window(cfg, c16.cache, q, cu, prefix, c16.d_table, most, window, sinks, out=out)
    torch.cuda.synchronize()
    assert torch.all(ws == 77) and torch.all(out == 9.0) and kv.get_device_status() == 0
    kv.prefill_window_fp8(cfg, c.cache, q, cu, prefix, c.d_table, n, window, sinks, out=out, workspace=ws)
    assert kv.get_device_status() == 0 and torch.all(out != 9.0) and not torch.all(ws == 77)


def test_prefill_longer_than_a_wait(kvattn_lib):
    """1.7 s of items without a row to zero (they end where a tile does), then one that has some: the role that zeroes
    them waits from the start to the end.  Keys of zeros and V of a power of two per dim make every sum exact."""
    kv = kvattn_lib
    keys, rows, block, d, heads = 2 ** 20, 190 * 256, 4096, 64, 128
    cfg = kv.make_config(heads, heads, d, kv.BF16)
    v = (2.0 ** (torch.arange(d) % 5)).to(torch.bfloat16)
    cache = kv.Cache(torch.zeros((2, heads, block, d), dtype=torch.bfloat16, device="cuda"),
                     v.expand(2, heads, block, d).contiguous().cuda())
    table = (torch.arange(keys // block, dtype=torch.int32) % 2).expand(2, -1).contiguous().cuda()
    q = torch.ones((rows + 1, heads, d), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, rows, rows + 1], dtype=torch.int32).cuda()
    prefix = torch.tensor([keys - rows, 0], dtype=torch.int32).cuda()
    out = torch.zeros_like(q)
    kv.prefill_window(cfg, cache, q, cu, prefix, table, rows, 2 ** 31 - 1, out=out)
    assert kv.get_device_status() == 0
    assert torch.all(out == v.cuda())


def test_prefill_of_a_very_long_sequence(kvattn_lib):
    """One row over 2^28 keys: refused where it sees more than 2^20 of them (the tensor cores' sums of equal V stop growing
    at 2^26), answered where it sees 2^20, and a chunk without rows is no error.  Keys of zeros and V of a power of two
    per dim make every sum exact."""
    kv = kvattn_lib
    keys, block, d = 2 ** 28, 4096, 64
    cfg = kv.make_config(1, 1, d, kv.BF16)
    v = (2.0 ** (torch.arange(d) % 5)).to(torch.bfloat16)
    cache = kv.Cache(torch.zeros((2, 1, block, d), dtype=torch.bfloat16, device="cuda"),
                     v.expand(2, 1, block, d).contiguous().cuda())
    table = (torch.arange(keys // block, dtype=torch.int32) % 2)[None].cuda()
    q = _q(1, (1, 1, d)).cuda()
    cu, prefix = torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([keys - 1], dtype=torch.int32).cuda()
    bad = kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    for window, sinks, status in ((2 ** 31 - 1, 0, bad), (2 ** 20 + 1, 0, bad), (2 ** 20, 4, bad), (1, 2 ** 20, bad),
                                  (2 ** 20, 0, 0), (2 ** 20 - 4, 4, 0), (1, 2 ** 20 - 1, 0)):
        out = torch.zeros_like(q)
        kv.prefill_window(cfg, cache, q, cu, prefix, table, 1, window, sinks, out=out)
        assert kv.get_device_status() == status, (window, sinks)
        assert torch.equal(out[0, 0].cpu(), torch.zeros_like(v) if status else v), (window, sinks)
    kv.prefill_window(cfg, cache, q, cu * 0, prefix, table, 1, 2 ** 31 - 1, out=out)
    assert kv.get_device_status() == 0


def test_prefill_fp8_of_a_very_long_sequence(kvattn_lib):
    """The same limit over an fp8 cache."""
    kv = kvattn_lib
    keys, block = 2 ** 20 + 16, 4096
    pool = torch.zeros((1, 1, block // 16, 4224), dtype=torch.uint8, device="cuda")
    pool[..., 2048:4096] = 0x38                                      # V = 1
    pool[..., 4096:] = torch.ones(32).view(torch.uint8).cuda()
    cfg = kv.make_config(4, 1, 128, kv.BF16)
    table = torch.zeros((1, -(-keys // block)), dtype=torch.int32, device="cuda")
    q = _q(1, (1, 4, 128)).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    for prefix, status in ((2 ** 20, kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]), (2 ** 20 - 1, 0)):
        out = torch.zeros_like(q)
        kv.prefill_window_fp8(cfg, kv.CacheFP8(pool, block), q, cu, torch.tensor([prefix], dtype=torch.int32).cuda(), table,
                              1, 2 ** 31 - 1, out=out)
        assert kv.get_device_status() == status
        assert torch.all(out == (0.0 if status else 1.0))


def test_python_integers_past_32_bits(kvattn_lib):
    """An integer that does not fit raises; its low 32 bits are not taken for it."""
    kv = kvattn_lib
    c = WindowCache(kv, "bf16", 2, 128, [40], [np.ones(40, bool)], seed=1)
    c8 = WindowCache(kv, "fp8", 2, 128, [40], [np.ones(40, bool)], seed=1)
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    q = _q(0, (1, 8, 128)).cuda()
    n = torch.tensor([40], dtype=torch.int32).cuda()
    cu, prefix = torch.tensor([0, 1], dtype=torch.int32).cuda(), n - 1
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 5.0)
    for given in (dict(out=out, workspace=ws), dict(out=out), {}):
        for cache, dec, pre in ((c.cache, kv.decode_window, kv.prefill_window),
                                (c8.cache, kv.decode_window_fp8, kv.prefill_window_fp8)):
            more = {k: v for k, v in given.items() if k == "out" or pre is kv.prefill_window_fp8}
            for wrong in (2 ** 32 + 16, 2 ** 31, -2 ** 32 + 16):
                for name in ("max_seq_len", "window", "num_sinks", "num_splits"):
                    with pytest.raises(ValueError, match=name):
                        dec(cfg, cache, q, c.d_table, n, **{**dict(max_seq_len=40, window=16, num_sinks=2), name: wrong}, **given)
                for name in ("max_q_len", "window", "num_sinks"):
                    with pytest.raises(ValueError, match=name):
                        pre(cfg, cache, q, cu, prefix, c.d_table, **{**dict(max_q_len=1, window=16, num_sinks=2), name: wrong},
                            **more)
            with pytest.raises(TypeError):
                dec(cfg, cache, q, c.d_table, n, 40, 16.0, **given)
    torch.cuda.synchronize()
    assert torch.all(out == 5.0)
    a = kv.decode_window(cfg, c.cache, q, c.d_table, n, np.int64(40), np.int32(16), 2)
    assert torch.equal(a, kv.decode_window(cfg, c.cache, q, c.d_table, n, 40, 16, 2, out=out, workspace=ws))


def test_calls_without_the_extension_module(kvattn_lib, monkeypatch):
    """The general way of marshalling gives what the extension module's gives."""
    kv = kvattn_lib
    c = WindowCache(kv, "bf16", 2, 128, [40], [np.ones(40, bool)], seed=1)
    c8 = WindowCache(kv, "fp8", 2, 128, [40], [np.ones(40, bool)], seed=1)
    cfg, form = kv.make_config(8, 2, 128, kv.BF16), kv.make_rotary("half")
    q, k = _q(0, (1, 8, 128)).cuda(), _q(1, (1, 2, 128)).cuda()
    n = torch.tensor([40], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()

    def calls():
        out = []
        for cache, app, dec, pre, ws in (
                (c.cache, kv.rotary_append, kv.decode_window, kv.prefill_window, {}),
                (c8.cache, kv.rotary_append_fp8, kv.decode_window_fp8, kv.prefill_window_fp8,
                 dict(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")))):
            r, a, b = (torch.zeros_like(q) for _ in range(3))
            app(cfg, form, cache, q, k, k, n - 1, n * 0, c.d_table if cache is c.cache else c8.d_table, q_out=r)
            table = c.d_table if cache is c.cache else c8.d_table
            dec(cfg, cache, r, table, n, 40, 16, 2, out=a, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
            pre(cfg, cache, r, cu, n - 1, table, 1, 16, 2, out=b, **ws)
            out += [r, a, b]
        return out

    calls()
    fast = calls()
    monkeypatch.setattr(kv, "_marshal", kv._General)
    slow = calls()
    monkeypatch.setattr(kv, "_raw_stream", None)          # as in a process that never had it
    slow += calls()
    assert kv.get_device_status() == 0
    for x, y in zip(fast + fast, slow):
        assert torch.equal(x, y) and x.abs().sum() > 0


def _decode_call(kv, dtype, hq, batch, keys, splits=0):
    """A decode_window call: sequences of one length, a cache larger than L2."""
    cfg = kv.make_config(hq, 1, 128, kv.F32 if dtype == "f32" else kv.BF16)
    t = TORCH_DT["f32" if dtype == "f32" else "bf16"]
    block = 256
    cache = kv.Cache(*(torch.zeros((batch * keys // block, 1, block, 128), dtype=t, device="cuda") for _ in range(2)))
    table = torch.arange(batch * keys // block, dtype=torch.int32, device="cuda").view(batch, -1)
    lens = torch.full((batch,), keys, dtype=torch.int32, device="cuda")
    q = torch.ones((batch, hq, 128), dtype=t, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(max(256, kv.decode_window_workspace_size(cfg, batch, keys, keys, 0, splits)), dtype=torch.uint8,
                     device="cuda")
    return lambda: kv.decode_window(cfg, cache, q, table, lens, keys, keys, out=out, workspace=ws, num_splits=splits)


def _times(*calls, n=20):
    """us of each call among others, timed in turn; the best of 7."""
    best = [float("inf")] * len(calls)
    for _ in range(8):  # (the first is a warm-up)
        for i, call in enumerate(calls):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(n):
                call()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b) * 1e3 / n)
    return best


@pytest.mark.parametrize("dtype,hq,few,more,keys", [("bf16", 4, 16, 20, 16384), ("bf16", 4, 16, 20, 32768),
                                                    ("f32", 1, 16, 20, 16384), ("bf16", 4, 38, 44, 16384)])
def test_fewer_sequences_take_no_longer(kvattn_lib, dtype, hq, few, more, keys):
    """A count of segments whose clusters are not resident at once, and a larger one whose smaller clusters are."""
    a, b = _times(*(_decode_call(kvattn_lib, dtype, hq, n, keys) for n in (few, more)))
    assert kvattn_lib.get_device_status() == 0
    print(f"{few}: {a:.1f} us, {more}: {b:.1f} us")
    assert a <= 1.04 * b, (a, b)


@pytest.mark.parametrize("dtype,hq,batch,keys", [("bf16", 1, 38, 16384), ("bf16", 4, 16, 32768), ("f32", 4, 16, 16384),
                                                 ("f32", 1, 16, 32768), ("bf16", 4, 8, 32768), ("bf16", 1, 1, 131072)])
def test_choice_of_the_decode_form(kvattn_lib, dtype, hq, batch, keys):
    """The library's own choice is no slower than the balanced stream with as many pieces as it would take (16)."""
    a, b = _times(*(_decode_call(kvattn_lib, dtype, hq, batch, keys, splits) for splits in (0, 16)))
    assert kvattn_lib.get_device_status() == 0
    print(f"{a:.1f} us, stream {b:.1f} us")
    assert a <= 1.09 * b, (a, b)


def test_first_cluster_in_a_capture(kvattn_lib):
    """A process whose first call of long windows, which takes several thread blocks a segment, is captured: what is asked
    of the runtime for it is no stream work, and its answer is the one outside a capture."""
    import os
    import subprocess
    import sys

    code = """
import sys
sys.path[:0] = [%r]
import torch, kv_cache_attention_rope_gb300 as kv
L, block = 16384, 256
table = torch.arange(L // block, dtype=torch.int32, device='cuda')[None]
n = torch.tensor([L], dtype=torch.int32, device='cuda')
ws = torch.empty(1 << 24, dtype=torch.uint8, device='cuda')
todo = []
for dtype, d in ((torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128)):
    cfg = kv.make_config(4, 1, d, kv.BF16 if dtype is torch.bfloat16 else kv.F32)
    cache = kv.Cache(*(torch.randn((L // block, 1, block, d), device='cuda').to(dtype) for _ in range(2)))
    q = torch.randn((1, 4, d), device='cuda').to(dtype)
    todo.append((kv.decode_window, cfg, cache, q, torch.zeros_like(q)))
pool = torch.randint(0, 64, (L // block, 1, block // 16, 4224), dtype=torch.uint8, device='cuda')
pool[..., 4096:] = torch.ones(32).view(torch.uint8).cuda()
q = torch.randn((1, 4, 128), device='cuda').to(torch.bfloat16)
todo.append((kv.decode_window_fp8, kv.make_config(4, 1, 128, kv.BF16), kv.CacheFP8(pool, block), q, torch.zeros_like(q)))
def calls():
    for f, cfg, cache, q, out in todo:
        f(cfg, cache, q, table, n, L, L, out=out, workspace=ws)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = [t[-1].clone() for t in todo]
calls()
torch.cuda.synchronize()
assert kv.get_device_status() == 0
for t, x in zip(todo, got):
    assert torch.equal(t[-1], x) and torch.isfinite(x).all() and x.abs().sum() > 0   # (the same sums in the same order)
print('captured')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code % root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 8, 2, 64), ("bf16", 2, 2, 128), ("f32", 8, 2, 128),
                                            ("fp8", 8, 2, 128)])
def test_seen_scores_of_minus_infinity(kvattn_lib, dtype, hq, hkv, d):
    """Keys whose score is -infinity (the newest one alone in its tile at 17, 33 and 4001 keys, and the first tile) weigh
    nothing, in every form of the decode and in the prefill."""
    kv = kvattn_lib
    lens = [17, 33, 40, 4001, 600]
    wanted = [np.ones(L, bool) for L in lens]
    c = WindowCache(kv, dtype, hkv, d, lens, wanted, seed=2)
    q = _q(3, (len(lens), hq, d), dtype).abs()
    low = [(0, 16), (1, 32), (2, 5), (3, 4000), *((4, t) for t in range(16))]
    for r, token in low:
        b, s = _at(c, r, token)
        if dtype == "fp8":  # codes of -1 with an infinite scale
            page = c.cache.pool[b, :, s // 16]
            page[:, 128 * (s % 16):128 * (s % 16) + 128] = 0xB8
            page[:, 4096 + 4 * (s % 16):4100 + 4 * (s % 16)] = torch.tensor([float("inf")]).view(torch.uint8).cuda()
        else:
            c.cache.k_pool[b, :, s, 0] = -float("inf")
        c.k[r][token, :, 0] = -np.inf
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    dec, win = (kv.decode_fp8, kv.decode_window_fp8) if dtype == "fp8" else (kv.decode, kv.decode_window)
    qd = q.cuda()
    got = {f"splits {s}": dec(cfg, c.cache, qd, c.d_table, n, max(lens), num_splits=s) for s in (0, 1, 3)}
    got |= {f"window, splits {s}": win(cfg, c.cache, qd, c.d_table, n, max(lens), 5000, num_splits=s) for s in (0, 1, 3)}
    if dtype != "f32":
        pre = kv.prefill_window_fp8 if dtype == "fp8" else kv.prefill_window
        got["prefill"] = pre(cfg, c.cache, qd, torch.arange(len(lens) + 1, dtype=torch.int32).cuda(), n - 1, c.d_table, 1, 5000)
    assert kv.get_device_status() == 0
    for r, L in enumerate(lens):
        want, mag = attend(q[r:r + 1].double().numpy(), c.k[r], c.v[r], wanted[r][None])
        for what, out in got.items():
            check_attention(f64(out)[r:r + 1], want, mag, dtype, f"{what}, length {L}")
