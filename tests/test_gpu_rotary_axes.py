"""GPU tests of rotary_append_axes and its fp8 form against the rotation in 64 bits.

Tolerances as test_gpu_rotary_append (the rotation is the same; only the position of a pair is its axis's).
"""
import numpy as np
import pytest
import torch

from oracle import fp8
from _window_support import TORCH_DT, speeds
from test_gpu_fp8 import unpack_rows
from test_gpu_rotary_append import Case, _close

pytestmark = pytest.mark.gpu


def axis_of_pairs(sections, order, pairs):
    if order == "sections":
        return np.repeat(np.arange(len(sections)), sections)
    n = len(sections)
    return np.array([i % n if i // n < sections[i % n] else 0 for i in range(pairs)])


def rotate_axes(x, positions, axis, f, rot, layout, amplitude=1.0):
    """x [T, H, D] in 64 bits, positions [A, T]: its rotation, and amplitude (|x0| + |x1|) of each element's pair."""
    y, size = x.copy(), np.zeros_like(x)
    a = positions.astype(np.float64)[axis].T * f
    c, s = (np.cos(a) * amplitude)[:, None], (np.sin(a) * amplitude)[:, None]
    n = rot // 2
    i0 = np.arange(n) if layout == "half" else 2 * np.arange(n)
    i1 = i0 + (n if layout == "half" else 1)
    x0, x1 = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = x0 * c - x1 * s, x0 * s + x1 * c
    size[..., i0] = size[..., i1] = amplitude * (np.abs(x0) + np.abs(x1))
    return y, size


FORMS = [("half", 128, "sections", [16, 24, 24]), ("adjacent", 128, "cyclic", [24, 20, 20]), ("half", 64, "sections", [0, 32]),
         ("half", 32, "cyclic", [6, 5, 5]), ("adjacent", 96, "sections", [1, 2, 0, 45]), ("half", 64, "cyclic", [32, 0, 0]),
         ("half", 64, "cyclic", [8, 8, 8, 8]), ("adjacent", 16, "sections", [8])]


def _positions(g, axes, T):
    p = g.integers(0, 5000, (axes, T)).astype(np.int32)
    p[:, 0] = 0
    p[:, 1] = np.arange(axes) * 131071 + 7
    return p


@pytest.mark.parametrize("layout,rot,order,sections", FORMS)
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("f32", 8, 2, 128), ("bf16", 12, 12, 64), ("f32", 12, 12, 64)])
def test_forms(kvattn_lib, dtype, hq, hkv, d, layout, rot, order, sections):
    kv = kvattn_lib
    if rot > d:
        pytest.skip("more rotated dims than the head has")
    c = Case(dtype, hq, hkv, d, [range(0, 19), [500], range(77, 90)], seed=rot + d)
    T = len(c.pos)
    p = _positions(np.random.default_rng(rot), len(sections), T)
    cfg = kv.make_config(hq, hkv, d, kv.BF16 if dtype == "bf16" else kv.F32)
    q_out = torch.empty((T, hq, d), dtype=TORCH_DT[dtype], device="cuda")
    cache = kv.Cache(*(x.cuda() for x in c.pools))
    kv.rotary_append_axes(cfg, kv.make_rotary(layout, rot), kv.make_axes(sections, order), cache, *c.split(kv),
                          torch.from_numpy(p).cuda(), *c.ints, q_out=q_out)
    assert kv.get_device_status() == 0
    assert torch.equal(c.qkv.cpu(), c.x)
    want, size = rotate_axes(c.x64[:, :hq + hkv], p, axis_of_pairs(sections, order, rot // 2), speeds(10000.0, rot), rot,
                             layout)
    _close(q_out.double().cpu().numpy(), want[:, :hq], size[:, :hq], dtype, "q")
    got_k, got_v = (x.double().cpu().numpy() for x in (cache.k_pool, cache.v_pool))
    _close(got_k[c.at], want[:, hq:], size[:, hq:], dtype, "k")
    assert np.array_equal(got_v[c.at], c.x64[:, hq + hkv:])
    for got, was in ((got_k, c.before[0]), (got_v, c.before[1])):
        got[c.at] = was[c.at]
        assert np.array_equal(got, was)


@pytest.mark.parametrize("tokens,hq,hkv,dtype,d", [(1, 12, 12, "f32", 64), (2500, 12, 12, "bf16", 64), (300, 32, 32, "f32", 128),
                                                   (1400, 64, 64, "bf16", 128)])
def test_launch_shapes(kvattn_lib, tokens, hq, hkv, dtype, d):
    """A warp, a thread block or several for a token; in place, speeds scaled, an amplitude."""
    kv = kvattn_lib
    c = Case(dtype, hq, hkv, d, [range(tokens)], seed=tokens)
    n = d // 2
    sections = [n - 2 * (n // 3), n // 3, n // 3]
    p = np.random.default_rng(1).integers(0, 3000, (3, tokens)).astype(np.int32)
    cfg = kv.make_config(hq, hkv, d, kv.BF16 if dtype == "bf16" else kv.F32)
    form = kv.make_rotary("half", 0, "linear", factor=4.0, amplitude=1.25)
    cache = kv.Cache(*(x.cuda() for x in c.pools))
    kv.rotary_append_axes(cfg, form, kv.make_axes(sections), cache, *c.split(kv), torch.from_numpy(p).cuda(), *c.ints)
    assert kv.get_device_status() == 0
    want, size = rotate_axes(c.x64[:, :hq + hkv], p, axis_of_pairs(sections, "sections", n),
                             speeds(10000.0, d, "linear", 4.0), d, "half", 1.25)
    got = c.qkv.double().cpu().numpy().reshape(c.x64.shape)
    _close(got[:, :hq], want[:, :hq], size[:, :hq], dtype, "q")
    assert np.array_equal(got[:, hq:], c.x64[:, hq:])
    _close(cache.k_pool.double().cpu().numpy()[c.at], want[:, hq:], size[:, hq:], dtype, "k")


@pytest.mark.parametrize("fp8_cache", [False, True])
def test_axes_alike_are_rotary_append(kvattn_lib, fp8_cache):
    """Text: every axis at the slot's position gives rotary_append's bits."""
    kv = kvattn_lib
    c = Case("bf16", 32, 8, 128, [range(100, 164), [7000]], block=32, seed=3)
    cfg, form = kv.make_config(32, 8, 128, kv.BF16), kv.make_rotary("half", 64)
    got = []
    for axes in (False, True):
        q_out = torch.empty((len(c.pos), 32, 128), dtype=torch.bfloat16, device="cuda")
        if fp8_cache:
            cache = kv.CacheFP8(torch.zeros((c.nb, 8, 2, 4224), dtype=torch.uint8, device="cuda"), 32)
        else:
            cache = kv.Cache(*(x.cuda() for x in c.pools))
        if axes:
            call = kv.rotary_append_axes_fp8 if fp8_cache else kv.rotary_append_axes
            call(cfg, form, kv.make_axes([12, 10, 10], "cyclic"), cache, *c.split(kv), c.ints[0].expand(3, -1).contiguous(),
                 *c.ints, q_out=q_out)
        else:
            (kv.rotary_append_fp8 if fp8_cache else kv.rotary_append)(cfg, form, cache, *c.split(kv), *c.ints, q_out=q_out)
        got.append([q_out] + ([cache.pool] if fp8_cache else [cache.k_pool, cache.v_pool]))
    assert kv.get_device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_fp8_slots(kvattn_lib):
    """Rows go to their slots, wherever their positions are: V bit for bit, K within half an e4m3 step of the rotation."""
    kv = kvattn_lib
    c = Case("bf16", 32, 8, 128, [range(3, 40), [77], range(160, 176)], block=32, seed=4)
    T = len(c.pos)
    p = np.random.default_rng(4).integers(0, 100000, (3, T)).astype(np.int32)
    cfg = kv.make_config(32, 8, 128, kv.BF16)
    cache = kv.CacheFP8(torch.zeros((c.nb, 8, 2, 4224), dtype=torch.uint8, device="cuda"), 32)
    q_out = torch.empty((T, 32, 128), dtype=torch.bfloat16, device="cuda")
    kv.rotary_append_axes_fp8(cfg, kv.make_rotary("half"), kv.make_axes([16, 24, 24]), cache, *c.split(kv),
                              torch.from_numpy(p).cuda(), *c.ints, q_out=q_out)
    assert kv.get_device_status() == 0
    want, size = rotate_axes(c.x64[:, :40], p, axis_of_pairs([16, 24, 24], "sections", 64), speeds(10000.0, 128), 128, "half")
    _close(q_out.double().cpu().numpy(), want[:, :32], size[:, :32], "bf16", "q")
    ck, sk, cv, sv = unpack_rows(cache.pool.cpu().numpy(), c.at[0], c.at[2])
    codes, scales = fp8.quantize_rows(c.x64[:, 40:])
    assert np.array_equal(sv, scales) and np.array_equal(fp8.e4m3_decode(cv), fp8.e4m3_decode(codes))
    wk, wsize = want[:, 32:], size[:, 32:]
    row = 2.0 ** -8 * (np.abs(wk) + 2.0 ** -21 * wsize) + 2.0 ** -21 * wsize
    step = np.maximum(2.0 ** -4 * (np.abs(wk) + row), 2.0 ** -10 * sk[..., None])
    assert np.all(np.abs(fp8.dequantize_rows(ck, sk) - wk) <= row + step * (1 + 2.0 ** -20) + 2.0 ** -22 * np.abs(wk))


@pytest.mark.parametrize("fp8_cache", [False, True])
def test_bad_tokens(kvattn_lib, fp8_cache):
    """A token with a negative position on some axis, a bad slot, row or block is skipped whole."""
    kv = kvattn_lib
    c = Case("bf16", 8, 2, 128, [range(0, 6), range(20, 23)], seed=9)
    T = len(c.pos)
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    if fp8_cache:
        cache = kv.CacheFP8(torch.zeros((c.nb, 2, 1, 4224), dtype=torch.uint8, device="cuda"))
    else:
        cache = kv.Cache(*(x.cuda() for x in c.pools))
    p = torch.zeros((3, T), dtype=torch.int32, device="cuda")
    slots, seq, table = (t.clone() for t in c.ints)
    slots[0], seq[1], slots[2], p[2, 3], seq[4] = -1, 2, 10 ** 6, -1, -3
    q_out = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    call = kv.rotary_append_axes_fp8 if fp8_cache else kv.rotary_append_axes
    call(cfg, kv.make_rotary("half"), kv.make_axes([16, 24, 24]), cache, *c.split(kv), p, slots, seq, table, q_out=q_out)
    assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    got = q_out.float().cpu()
    assert torch.all(got[:5] == 7.0) and not torch.any(got[5:] == 7.0)
    for i in range(5):  # its slot as it was
        b, s = c.at[0][i], c.at[2][i]
        if not fp8_cache:
            assert torch.equal(cache.k_pool[b, :, s].cpu(), c.pools[0][b, :, s])
            assert torch.equal(cache.v_pool[b, :, s].cpu(), c.pools[1][b, :, s])
        else:
            ck, sk, cv, sv = unpack_rows(cache.pool.cpu().numpy(), c.at[0][i:i + 1], c.at[2][i:i + 1])
            assert not ck.any() and not cv.any() and not sk.any() and not sv.any(), i


def test_captured_and_far(kvattn_lib):
    """Captured and replayed over new positions; positions up to the last of 32 bits."""
    kv = kvattn_lib
    c = Case("bf16", 32, 8, 128, [range(0, 50), [4000]], seed=6)
    T = len(c.pos)
    cfg, form, axes = kv.make_config(32, 8, 128, kv.BF16), kv.make_rotary("half"), kv.make_axes([16, 24, 24])
    cache = kv.Cache(*(x.cuda() for x in c.pools))
    p = torch.zeros((3, T), dtype=torch.int32, device="cuda")
    q_out = torch.zeros((T, 32, 128), dtype=torch.bfloat16, device="cuda")
    args = (cfg, form, axes, cache, *c.split(kv), p, *c.ints)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.rotary_append_axes(*args, q_out=q_out)
    graph.replay()
    first = q_out.clone()
    p.copy_(torch.from_numpy(np.random.default_rng(2).integers(0, 2 ** 31 - 1, (3, T)).astype(np.int32)))
    graph.replay()
    got = q_out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv.rotary_append_axes(*args, q_out=q_out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, q_out) and not torch.equal(got, first)
    assert kv.get_device_status() == 0
    from fractions import Fraction
    x, pos = c.x64[:2, :32], p.cpu().numpy()
    for t in range(2):  # angles of far positions from the speeds held as exact fractions of a turn
        for i in (0, 1, 5, 20, 63):
            a = 0 if i < 16 else 1 if i < 40 else 2
            from decimal import Decimal, getcontext
            getcontext().prec = 50
            two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")
            turns = (Decimal(10000) ** (Decimal(-2 * i) / Decimal(128))) / two_pi
            u = Fraction(Decimal(int(pos[a, t])) * turns)
            ang = float(u - (u.numerator // u.denominator)) * 2 * np.pi
            x0, x1 = x[t, :, i], x[t, :, i + 64]
            w = x0 * np.cos(ang) - x1 * np.sin(ang)
            bound = 2.0 ** -8 * (np.abs(w) + 2.0 ** -21 * (np.abs(x0) + np.abs(x1))) + 2.0 ** -20 * (np.abs(x0) + np.abs(x1))
            assert np.all(np.abs(got[t, :, i].double().cpu().numpy() - w) <= bound), (t, i)


def test_refusals_of_tensors(kvattn_lib):
    kv = kvattn_lib
    c = Case("bf16", 8, 2, 128, [range(4)], seed=1)
    cfg, form, axes = kv.make_config(8, 2, 128, kv.BF16), kv.make_rotary("half"), kv.make_axes([16, 24, 24])
    cache = kv.Cache(*(x.cuda() for x in c.pools))
    q, k, v = c.split(kv)
    p = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    for wrong in ((p[:2], *c.ints), (p.t().contiguous(), *c.ints), (p.long(), *c.ints), (p, c.ints[0][:2], *c.ints[1:]),
                  (p, c.ints[0].cpu(), *c.ints[1:])):
        with pytest.raises((TypeError, ValueError)):
            kv.rotary_append_axes(cfg, form, axes, cache, q, k, v, *wrong)
    with pytest.raises(kv.KvattnError):
        kv.rotary_append_axes(cfg, form, kv.make_axes([16, 24, 25]), cache, q, k, v, p, *c.ints)
