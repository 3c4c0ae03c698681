"""GPU tests of rotary_append and rotary_append_fp8 against the rotation in 64 bits.

Tolerance: a stored element is the fp32 rotation rounded once, so it is off by half a step of its type (relative
2^-8 for bf16, 2^-24 for fp32) plus the rotation's own error.  That is at most 8 * 2^-24 = 2^-21 of a(|x0| + |x1|):
the remainder's rounding (pi/4 * 2^-24), sincospi (2 ulp, 2^-23), the amplitude's product, the element's product and
its fma (2^-24 each) sum to less than 7 * 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import fp8
from _window_support import HALF_STEP, TORCH_DT, rotate, speeds
from test_gpu_fp8 import unpack_rows

pytestmark = pytest.mark.gpu


def _close(got, want, size, dtype, what):
    bound = (np.abs(want) + 2.0 ** -21 * size) * HALF_STEP[dtype] + 2.0 ** -21 * size
    over = np.abs(got - want) - bound
    assert np.all(over <= 0), f"{what}: {over.max():.3e} past the bound"


class Case:
    """Tokens of several sequences in a random order, over a pool filled with a pattern."""

    def __init__(self, dtype, hq, hkv, d, positions, block=16, seed=0, fused=True):
        g = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.block, self.dtype = hq, hkv, d, block, dtype
        t = TORCH_DT[dtype]
        seqs = [(r, p) for r, run in enumerate(positions) for p in run]
        seqs = [seqs[i] for i in g.permutation(len(seqs))]
        self.seq = np.array([s for s, _ in seqs], np.int32)
        self.pos = np.array([p for _, p in seqs], np.int32)
        width = max(max(run) for run in positions) // block + 1
        used = sorted({(s, p // block) for s, p in seqs})
        self.nb = len(used) + 2
        self.table = np.full((len(positions), width), -1, np.int32)
        for (s, c), b in zip(used, g.permutation(self.nb)):
            self.table[s, c] = b
        T = len(seqs)
        self.x = torch.from_numpy(g.standard_normal((T, (hq + 2 * hkv) * d))).to(t)
        self.x64 = self.x.double().numpy().reshape(T, hq + 2 * hkv, d)
        self.qkv = self.x.cuda()
        self.pools = [torch.from_numpy(g.standard_normal((self.nb, hkv, block, d))).to(t) for _ in range(2)]
        self.before = [p.double().numpy() for p in self.pools]
        self.ints = [torch.from_numpy(a).cuda() for a in (self.pos, self.seq, self.table)]
        self.at = (self.table[self.seq, self.pos // block], slice(None), self.pos % block)

    def split(self, kv, fused=True):
        q, k, v = kv.split_qkv(self.qkv, self.hq, self.hkv, self.d)
        return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


FORMS = [("half", 0, "none", {}), ("adjacent", 0, "none", {}), ("half", 32, "linear", dict(factor=4.0)),
         ("adjacent", 48, "base", dict(factor=8.0)),
         ("half", 0, "parts", dict(factor=8.0, original_len=4096.0, low=1.0, high=32.0, amplitude=1.1875)),
         ("adjacent", 16, "parts", dict(factor=2.0, original_len=512.0, low=0.0, high=4.0, amplitude=0.5))]


@pytest.mark.parametrize("layout,rot,scaling,more", FORMS)
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("f32", 12, 12, 64), ("bf16", 8, 1, 64),
                                            ("f32", 8, 2, 128)])
def test_forms(kvattn_lib, dtype, hq, hkv, d, layout, rot, scaling, more):
    kv = kvattn_lib
    c = Case(dtype, hq, hkv, d, [range(0, 17), [5], range(4090, 4100), [131071], [1000003]], seed=d + hq)
    cfg = kv.make_config(hq, hkv, d, kv.BF16 if dtype == "bf16" else kv.F32, rope_base=10000.0)
    q, k, v = c.split(kv)
    q_out = torch.empty((len(c.pos), hq, d), dtype=TORCH_DT[dtype], device="cuda")
    cache = kv.Cache(*(p.cuda() for p in c.pools))
    kv.rotary_append(cfg, kv.make_rotary(layout, rot, scaling, **more), cache, q, k, v, *c.ints, q_out=q_out)
    assert kv.get_device_status() == 0
    assert torch.equal(c.qkv.cpu(), c.x), "the projection output was written"
    more = dict(more)
    amplitude = more.pop("amplitude", 1.0)
    R = rot or d
    want, size = rotate(c.x64[:, :hq + hkv], c.pos, speeds(10000.0, R, scaling, **more), R, layout, amplitude)
    _close(q_out.double().cpu().numpy(), want[:, :hq], size[:, :hq], dtype, "q")
    got_k, got_v = (p.double().cpu().numpy() for p in (cache.k_pool, cache.v_pool))
    _close(got_k[c.at], want[:, hq:], size[:, hq:], dtype, "k")
    assert np.array_equal(got_v[c.at], c.x64[:, hq + hkv:])
    for got, was in ((got_k, c.before[0]), (got_v, c.before[1])):  # every other slot as it was
        got[c.at] = was[c.at]
        assert np.array_equal(got, was)


@pytest.mark.parametrize("block", [16, 48, 1040])
def test_in_place_dense_and_block_sizes(kvattn_lib, block):
    kv = kvattn_lib
    c = Case("bf16", 16, 4, 128, [range(30, 75), [999]], block=block, seed=block)
    cfg = kv.make_config(16, 4, 128, kv.BF16)
    q, k, v = c.split(kv, fused=False)
    cache = kv.Cache(*(p.cuda() for p in c.pools))
    kv.rotary_append(cfg, kv.make_rotary("half"), cache, q, k, v, *c.ints)
    assert kv.get_device_status() == 0
    want, size = rotate(c.x64[:, :20], c.pos, speeds(10000.0, 128), 128, "half", 1.0)
    _close(q.double().cpu().numpy(), want[:, :16], size[:, :16], "bf16", "q in place")
    _close(cache.k_pool.double().cpu().numpy()[c.at], want[:, 16:], size[:, 16:], "bf16", "k")


@pytest.mark.parametrize("dtype,hq,hkv,tokens,layout,rot", [
    ("f32", 32, 32, 5, "half", 0), ("f32", 32, 32, 300, "adjacent", 64), ("f32", 32, 32, 700, "half", 16),
    ("f32", 32, 32, 1300, "half", 0), ("bf16", 128, 16, 7, "adjacent", 0), ("bf16", 64, 64, 1301, "half", 96),
    ("f32", 32, 8, 40, "half", 0)])
def test_large_tokens(kvattn_lib, dtype, hq, hkv, tokens, layout, rot):
    """Tokens of many heads, few and many of them: a token's heads may be several thread blocks' work.  In place."""
    kv = kvattn_lib
    c = Case(dtype, hq, hkv, 128, [range(50, 50 + tokens - tokens // 2), range(tokens // 2)], seed=tokens)
    cfg = kv.make_config(hq, hkv, 128, kv.BF16 if dtype == "bf16" else kv.F32)
    cache = kv.Cache(*(p.cuda() for p in c.pools))
    kv.rotary_append(cfg, kv.make_rotary(layout, rot), cache, *c.split(kv), *c.ints)
    assert kv.get_device_status() == 0
    R = rot or 128
    want, size = rotate(c.x64[:, :hq + hkv], c.pos, speeds(10000.0, R), R, layout, 1.0)
    got = c.qkv.double().cpu().numpy().reshape(c.x64.shape)
    _close(got[:, :hq], want[:, :hq], size[:, :hq], dtype, "q")
    assert np.array_equal(got[:, hq:], c.x64[:, hq:]), "k or v of the projection output was written"
    got_k, got_v = (p.double().cpu().numpy() for p in (cache.k_pool, cache.v_pool))
    _close(got_k[c.at], want[:, hq:], size[:, hq:], dtype, "k")
    assert np.array_equal(got_v[c.at], c.x64[:, hq + hkv:])


def test_adjacent_whole_head_is_rope_append(kvattn_lib):
    """The form rope_append has: its correctly rounded values, up to the fp32 rotation's error."""
    kv = kvattn_lib
    c = Case("bf16", 32, 8, 128, [range(100, 164), [7000]], seed=3)
    cfg = kv.make_config(32, 8, 128, kv.BF16)
    got = []
    for call in (lambda *a, **k: kv.rotary_append(cfg, kv.make_rotary(), *a, **k),
                 lambda *a, **k: kv.rope_append(cfg, *a, **k)):
        cache = kv.Cache(*(p.cuda() for p in c.pools))
        q_out = torch.empty((len(c.pos), 32, 128), dtype=torch.bfloat16, device="cuda")
        call(cache, *c.split(kv), *c.ints, q_out=q_out)
        got.append([t.double().cpu().numpy() for t in (q_out, cache.k_pool[c.at[0], :, c.at[2]], cache.v_pool)])
    assert np.array_equal(got[0][2], got[1][2])
    _, size = rotate(c.x64[:, :40], c.pos, speeds(10000.0, 128), 128, "adjacent", 1.0)
    for i, s in ((0, size[:, :32]), (1, size[:, 32:])):
        # two roundings of values 2^-21 size apart: at most a whole step apart, and only beside a border
        assert np.all(np.abs(got[0][i] - got[1][i]) <= 2.0 ** -7 * np.abs(got[1][i]) + 2.0 ** -20 * s)
        assert (got[0][i] != got[1][i]).mean() < 0.002


def test_passed_through_dims_and_bad_tokens(kvattn_lib):
    """Infinities and NaN past rotary_dim are copied; a token with a bad position, row or block is skipped whole."""
    kv = kvattn_lib
    c = Case("bf16", 8, 2, 64, [range(0, 6), range(20, 23)], seed=9)
    with torch.no_grad():
        c.qkv.view(-1, 12, 64)[:, :, 32:] = float("inf")
        c.qkv.view(-1, 12, 64)[:, :, 40] = float("nan")
    cfg = kv.make_config(8, 2, 64, kv.BF16)
    cache = kv.Cache(*(p.cuda() for p in c.pools))
    q_out = torch.full((len(c.pos), 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pos, seq, table = (t.clone() for t in c.ints)
    pos[0], seq[1], pos[2] = -1, 2, 10 ** 6
    kv.rotary_append(cfg, kv.make_rotary("half", 32), cache, *c.split(kv), pos, seq, table, q_out=q_out)
    assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    got = q_out.float().cpu()
    assert torch.all(got[:3] == 7.0)
    x = c.qkv.float().cpu().view(-1, 12, 64)
    assert torch.equal(torch.nan_to_num(got[3:, :, 32:], nan=-1.0), torch.nan_to_num(x[3:, :8, 32:], nan=-1.0))
    assert torch.isfinite(got[3:, :, :32]).all()
    k = cache.k_pool.float().cpu()
    for i in range(3):  # its slot as it was
        b, s = c.at[0][i], c.at[2][i]
        assert torch.equal(k[b, :, s], c.pools[0][b, :, s].float())


@pytest.mark.parametrize("tokens", [0, 1])
def test_few_tokens(kvattn_lib, tokens):
    kv = kvattn_lib
    c = Case("f32", 12, 12, 64, [[1023]], seed=2)
    cfg = kv.make_config(12, 12, 64, kv.F32)
    cache = kv.Cache(*(p.cuda() for p in c.pools))
    q, k, v = (t[:tokens] for t in c.split(kv))
    q_out = torch.zeros((tokens, 12, 64), device="cuda")
    kv.rotary_append(cfg, kv.make_rotary("half"), cache, q, k, v, c.ints[0][:tokens], c.ints[1][:tokens], c.ints[2],
                     q_out=q_out)
    assert kv.get_device_status() == 0
    if tokens:
        want, size = rotate(c.x64[:, :24], c.pos, speeds(10000.0, 64), 64, "half", 1.0)
        _close(q_out.double().cpu().numpy(), want[:, :12], size[:, :12], "f32", "q")
    else:
        assert torch.equal(cache.k_pool.cpu(), c.pools[0])


@pytest.mark.parametrize("layout,rot,hq,hkv", [("half", 0, 32, 8), ("half", 64, 32, 8), ("adjacent", 0, 32, 8),
                                               ("adjacent", 32, 32, 8), ("half", 0, 128, 16), ("adjacent", 96, 64, 16)])
def test_fp8_rows(kvattn_lib, layout, rot, hq, hkv):
    """Codes and scales of each row are the quantisation of a bf16 row within the rotation's bound: V's bit for bit,
    K's values within half an e4m3 step (2^-4 relative, 2^-10 of the scale's 448 below the normals) of it."""
    kv = kvattn_lib
    c = Case("bf16", hq, hkv, 128, [range(3, 40), [77], range(160, 176)], block=32, seed=4)
    cfg = kv.make_config(hq, hkv, 128, kv.BF16)
    cache = kv.CacheFP8(torch.zeros((c.nb, hkv, 2, 4224), dtype=torch.uint8, device="cuda"), 32)
    q_out = torch.empty((len(c.pos), hq, 128), dtype=torch.bfloat16, device="cuda")
    kv.rotary_append_fp8(cfg, kv.make_rotary(layout, rot), cache, *c.split(kv), *c.ints, q_out=q_out)
    assert kv.get_device_status() == 0
    R = rot or 128
    want, size = rotate(c.x64[:, :hq + hkv], c.pos, speeds(10000.0, R), R, layout, 1.0)
    _close(q_out.double().cpu().numpy(), want[:, :hq], size[:, :hq], "bf16", "q")
    ck, sk, cv, sv = unpack_rows(cache.pool.cpu().numpy(), c.at[0], c.at[2])
    codes, scales = fp8.quantize_rows(c.x64[:, hq + hkv:])
    assert np.array_equal(sv, scales)
    assert np.array_equal(fp8.e4m3_decode(cv), fp8.e4m3_decode(codes))
    wk, wsize = want[:, hq:], size[:, hq:]
    row = 2.0 ** -8 * (np.abs(wk) + 2.0 ** -21 * wsize) + 2.0 ** -21 * wsize       # the stored bf16 row
    amax = np.abs(wk).max(-1)
    # the scale: amax is of the bf16 row; amax / 448 is rounded to fp32
    assert np.all(np.abs(sk * 448.0 - amax) <= row.max(-1) + 2.0 ** -23 * amax)
    got = fp8.dequantize_rows(ck, sk)
    step = np.maximum(2.0 ** -4 * (np.abs(wk) + row), 2.0 ** -10 * sk[..., None])   # half a step of the code
    assert np.all(np.abs(got - wk) <= row + step * (1 + 2.0 ** -20) + 2.0 ** -22 * np.abs(wk))


def test_captured_and_on_another_stream(kvattn_lib):
    kv = kvattn_lib
    c = Case("bf16", 32, 8, 128, [range(0, 50), [4000]], seed=6)
    cfg = kv.make_config(32, 8, 128, kv.BF16)
    form = kv.make_rotary("half", 64, "linear", factor=2.0)
    cache = kv.Cache(*(p.cuda() for p in c.pools))
    q, k, v = c.split(kv)
    q_out = torch.zeros((len(c.pos), 32, 128), dtype=torch.bfloat16, device="cuda")
    kv.rotary_append(cfg, form, cache, q, k, v, *c.ints, q_out=q_out)
    first = [t.clone() for t in (q_out, cache.k_pool, cache.v_pool)]
    side = torch.cuda.Stream()
    for t in (q_out, cache.k_pool, cache.v_pool):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.rotary_append(cfg, form, cache, q, k, v, *c.ints, q_out=q_out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q_out, first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.rotary_append(cfg, form, cache, q, k, v, *c.ints, q_out=q_out)
    c.qkv.copy_(c.qkv.flip(0))  # the graph reads the new inputs
    graph.replay()
    got = q_out.clone()
    kv.rotary_append(cfg, form, cache, q, k, v, *c.ints, q_out=q_out)
    assert torch.equal(got, q_out) and not torch.equal(got, first[0])
    assert kv.get_device_status() == 0
