"""GPU tests of windowed decode and prefill attention against the formula in 64 bits.

Every slot that no query sees holds NaN and every block without a seen key is -1 in the table, so a key outside the
mask that reaches a result, or a block id read in vain, fails.  Tolerances: _window_support.check_attention.
"""
import numpy as np
import pytest
import torch

from _window_support import TORCH_DT, WindowCache, attend, check_attention, seen
from _gpu_support import f64

pytestmark = pytest.mark.gpu

ALL = 2 ** 31 - 1
LENS = [0, 1, 15, 16, 17, 31, 33, 64, 129, 500, 777]


def _q(g, shape, dtype):
    return torch.from_numpy(g.standard_normal(shape)).to(TORCH_DT["f32" if dtype == "f32" else "bf16"])


def _decode(kv, dtype, hq, hkv, d, lens, window, sinks, block=16, splits=0, seed=0):
    wanted = [seen([L - 1], L, window, sinks)[0] if L else np.zeros(0, bool) for L in lens]
    c = WindowCache(kv, dtype, hkv, d, lens, wanted, block=block, seed=seed)
    q = _q(np.random.default_rng(seed + 1), (len(lens), hq, d), dtype)
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_window_fp8 if dtype == "fp8" else kv.decode_window
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    call(cfg, c.cache, q.cuda(), c.d_table, torch.tensor(lens, dtype=torch.int32).cuda(), max(lens), window, sinks,
         out=out, num_splits=splits)
    assert kv.get_device_status() == 0
    got = f64(out)
    for r, L in enumerate(lens):
        want, mag = attend(q[r:r + 1].double().numpy(), c.k[r], c.v[r], wanted[r][None])
        check_attention(got[r:r + 1], want, mag, dtype, f"length {L}, window {window}, sinks {sinks}")
        if L == 0:
            assert np.all(got[r] == 0.0)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 0), (17, 16), (100, 4), (100, 17), (333, 40),
                                          (ALL, 0), (5, 600), (1, ALL)])
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 8, 8, 128), ("f32", 12, 12, 64),
                                            ("fp8", 16, 4, 128)])
@pytest.mark.parametrize("splits", [0, 3])
def test_decode_masks(kvattn_lib, dtype, hq, hkv, d, window, sinks, splits):
    """In one launch (splits 0: these are few keys) and over the balanced stream."""
    _decode(kvattn_lib, dtype, hq, hkv, d, LENS, window, sinks, splits=splits, seed=window % 97 + sinks % 89)


@pytest.mark.parametrize("dtype,hq,hkv,d,block", [("bf16", 64, 8, 128, 16), ("bf16", 8, 1, 128, 48), ("bf16", 4, 2, 64, 32),
                                                  ("bf16", 16, 2, 64, 16), ("bf16", 8, 4, 128, 16), ("f32", 32, 4, 128, 16),
                                                  ("f32", 8, 2, 64, 64), ("fp8", 8, 1, 128, 32), ("fp8", 64, 8, 128, 16)])
@pytest.mark.parametrize("splits", [0, 2])
def test_decode_heads_and_blocks(kvattn_lib, dtype, hq, hkv, d, block, splits):
    _decode(kvattn_lib, dtype, hq, hkv, d, LENS, 75, 5, block=block, splits=splits, seed=hq)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 1, 128), ("bf16", 4, 4, 64), ("fp8", 4, 1, 128), ("f32", 1, 1, 128),
                                            ("f32", 2, 1, 64), ("f32", 4, 1, 64), ("f32", 8, 1, 128), ("f32", 2, 1, 128)])
@pytest.mark.parametrize("lens,window", [([9000], 6000), ([1, 4000, 0, 2500, 16], 3000), ([300] * 40, 250),
                                         ([35, 0, 20] * 120, 34)])
def test_decode_clusters(kvattn_lib, dtype, hq, hkv, d, lens, window):
    """From several thread blocks per segment, and several rounds of 32 tiles per warp, to several segments a block."""
    _decode(kvattn_lib, dtype, hq, hkv, d, lens, window, 20, seed=len(lens))


@pytest.mark.parametrize("splits", [1, 2, 5, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_decode_splits(kvattn_lib, dtype, splits):
    _decode(kvattn_lib, dtype, 8, 2, 128, [3000, 0, 2200, 17, 801], 700, 33, splits=splits, seed=splits)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("f32", 12, 12, 64), ("bf16", 8, 2, 128), ("bf16", 8, 8, 64)])
@pytest.mark.parametrize("splits", [0, 2])
def test_decode_contiguous_cache(kvattn_lib, dtype, hq, hkv, d, splits):
    """One row per sequence, of a length that is no multiple of 16."""
    _decode(kvattn_lib, dtype, hq, hkv, d, [1, 777, 400, 775], 130, 3, block=777, splits=splits, seed=5)


def test_decode_one_and_many_sequences(kvattn_lib):
    _decode(kvattn_lib, "bf16", 32, 8, 128, [5000], 128, 4, seed=1)
    _decode(kvattn_lib, "bf16", 8, 2, 128, [(37 * i) % 400 for i in range(301)], 60, 2, seed=2)


def test_decode_whole_window_is_decode(kvattn_lib):
    kv = kvattn_lib
    lens = [900, 16, 333]
    c = WindowCache(kv, "bf16", 8, 128, lens, [np.ones(L, bool) for L in lens], seed=8)
    q = _q(np.random.default_rng(3), (3, 32, 128), "bf16").cuda()
    cfg = kv.make_config(32, 8, 128, kv.BF16)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    a = kv.decode_window(cfg, c.cache, q, c.d_table, n, 900, ALL, num_splits=1)
    b = kv.decode(cfg, c.cache, q, c.d_table, n, 900, num_splits=1)
    # the same keys in the same 16-key tiles, whatever shares the work: the weights and sums differ by the running
    # maximum's choice only, so each within the attention bound of the formula
    for r, L in enumerate(lens):
        want, mag = attend(f64(q[r:r + 1]), c.k[r], c.v[r], np.ones((1, L), bool))
        for got in (a, b):
            check_attention(f64(got)[r:r + 1], want, mag, "bf16", "whole window")


def test_decode_bad_lengths_and_blocks(kvattn_lib):
    kv = kvattn_lib
    lens = [40, 40, 40]
    c = WindowCache(kv, "bf16", 2, 128, lens, [np.ones(40, bool)] * 3, seed=8)
    q = _q(np.random.default_rng(3), (3, 8, 128), "bf16").cuda()
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    n = torch.tensor([40, 41, -1], dtype=torch.int32).cuda()
    out = kv.decode_window(cfg, c.cache, q, c.d_table, n, 40, 16, 2)
    assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    assert torch.all(out[1:] == 0) and torch.isfinite(out[0]).all()
    table = c.d_table.clone()
    table[0, 2] = 10 ** 6
    kv.decode_window(cfg, c.cache, q[:1], table, n[:1], 40, 8, 2)
    assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]


def _chunk_case(kv, dtype, hq, hkv, d, chunks, window, sinks, block=16, seed=0, spare_rows=0):
    """(prefix, queries) chunks: the call's output and the reference rows."""
    lens = [p + n for p, n in chunks]
    masks = [seen(range(p, p + n), p + n, window, sinks) for p, n in chunks]
    wanted = [m.any(0) if len(m) else np.zeros(L, bool) for m, L in zip(masks, lens)]
    c = WindowCache(kv, dtype, hkv, d, lens, wanted, block=block, seed=seed)
    cu = np.concatenate([[0], np.cumsum([n for _, n in chunks])]).astype(np.int32)
    q = _q(np.random.default_rng(seed + 1), (int(cu[-1]) + spare_rows, hq, d), dtype)
    cfg = kv.make_config(hq, hkv, d, kv.BF16)
    call = kv.prefill_window_fp8 if dtype == "fp8" else kv.prefill_window
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    call(cfg, c.cache, q.cuda(), torch.from_numpy(cu).cuda(),
         torch.tensor([p for p, _ in chunks], dtype=torch.int32).cuda(), c.d_table, max(n for _, n in chunks), window,
         sinks, out=out)
    assert kv.get_device_status() == 0
    return c, q, cu, masks, f64(out)


def _prefill(kv, dtype, hq, hkv, d, chunks, window, sinks, step=1, **more):
    c, q, cu, masks, got = _chunk_case(kv, dtype, hq, hkv, d, chunks, window, sinks, **more)
    for i, (p, n) in enumerate(chunks):
        rows = np.unique(np.concatenate([np.arange(0, n, step), np.arange(max(0, n - 2), n)]))
        want, mag = attend(q[cu[i] + rows].double().numpy(), c.k[i], c.v[i], masks[i][rows])
        check_attention(got[cu[i] + rows], want, mag, dtype, f"chunk {p}+{n}, window {window}, sinks {sinks}")
    assert np.all(got[cu[-1]:] == 9.0), "rows behind the last chunk were written"


CHUNKS = [(0, 1), (0, 200), (17, 130), (300, 64), (1000, 300), (5, 0), (255, 257)]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (100, 4), (128, 16), (129, 17), (300, 140), (700, 1),
                                          (ALL, 0), (20, 2000)])
def test_prefill_masks(kvattn_lib, window, sinks):
    _prefill(kvattn_lib, "bf16", 4, 2, 128, CHUNKS, window, sinks, step=5, seed=window % 97, spare_rows=5)


@pytest.mark.parametrize("window,sinks", [(1, 1), (100, 4), (129, 40), (ALL, 0), (30, 600)])
def test_prefill_masks_fp8(kvattn_lib, window, sinks):
    _prefill(kvattn_lib, "fp8", 8, 2, 128, CHUNKS, window, sinks, step=7, block=32, seed=window % 97, spare_rows=5)


@pytest.mark.parametrize("dtype,hq,hkv,d,block", [("bf16", 12, 12, 64, 16), ("bf16", 16, 2, 64, 128), ("bf16", 8, 1, 128, 48),
                                                  ("bf16", 4, 4, 128, 1040), ("fp8", 16, 4, 128, 16)])
def test_prefill_heads_and_blocks(kvattn_lib, dtype, hq, hkv, d, block):
    _prefill(kvattn_lib, dtype, hq, hkv, d, [(700, 290), (0, 77), (64, 1)], 150, 5, step=11, block=block, seed=hq)


@pytest.mark.parametrize("scale,k_scale", [(2.0 ** -30, 1.0), (2.0 ** 20, 2.0 ** 7), (1.0, 2.0 ** -14)])
def test_prefill_fp8_k_and_v_of_any_size(kvattn_lib, scale, k_scale):
    """K and V far outside f16's range, V's size differing by head and token, q as small or large as K is large or small."""
    kv = kvattn_lib
    lens, window, sinks = [300, 70], 120, 4
    chunks = [(100, 200), (0, 70)]
    masks = [seen(range(p, p + n), p + n, window, sinks) for p, n in chunks]
    c = WindowCache(kv, "fp8", 2, 128, lens, [m.any(0) for m in masks], seed=3)
    pool = c.cache.pool
    scales = pool[..., 4160:].contiguous().view(torch.float32)                       # [blocks, heads, 1, 16]
    times = scale * 2.0 ** torch.tensor([0.0, 7.0], device="cuda")[:, None, None]    # by head ...
    times = times * 2.0 ** -(torch.arange(16, device="cuda") % 4).float()            # ... and by token
    pool[..., 4160:] = (scales * times).view(torch.uint8)
    pool[..., 4096:4160] = (pool[..., 4096:4160].contiguous().view(torch.float32) * k_scale).view(torch.uint8)
    c.k = [x * k_scale for x in c.k]
    c.v = [x * times[:, 0].double().cpu().numpy().T[np.arange(len(x)) % 16][:, :, None] for x in c.v]
    q = _q(np.random.default_rng(1), (270, 8, 128), "bf16") / k_scale
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    out = kv.prefill_window_fp8(cfg, c.cache, q.cuda(), torch.tensor([0, 200, 270], dtype=torch.int32).cuda(),
                                torch.tensor([100, 0], dtype=torch.int32).cuda(), c.d_table, 200, window, sinks)
    assert kv.get_device_status() == 0
    for i, (a, b) in enumerate([(0, 200), (200, 270)]):
        want, mag = attend(q[a:b].double().numpy(), c.k[i], c.v[i], masks[i])
        check_attention(f64(out)[a:b], want, mag, "fp8", f"chunk {i}")


def test_prefill_more_items_than_processors(kvattn_lib):
    chunks = [(3000, 512), (0, 300), (700, 17), (1500, 512), (64, 256), (2222, 1)]
    _prefill(kvattn_lib, "bf16", 32, 8, 128, chunks, 600, 4, step=37, seed=6)


def test_prefill_one_query_is_decode(kvattn_lib):
    """A chunk of one row and decode_window see the same keys: both within the bound."""
    kv = kvattn_lib
    lens = [1, 600, 129, 700]
    wanted = [seen([L - 1], L, 100, 4)[0] for L in lens]
    c = WindowCache(kv, "bf16", 2, 128, lens, wanted, seed=4)
    q = _q(np.random.default_rng(5), (4, 8, 128), "bf16").cuda()
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    a = kv.decode_window(cfg, c.cache, q, c.d_table, n, 700, 100, 4)
    b = kv.prefill_window(cfg, c.cache, q, torch.arange(5, dtype=torch.int32).cuda(), n - 1, c.d_table, 1, 100, 4)
    assert kv.get_device_status() == 0
    for r in range(4):
        want, mag = attend(f64(q[r:r + 1]), c.k[r], c.v[r], wanted[r][None])
        for got in (a, b):
            check_attention(f64(got)[r:r + 1], want, mag, "bf16", f"length {lens[r]}")


def test_prefill_growing_scores(kvattn_lib):
    """Scores that grow along the keys: the running maximum moves by more than its slack in most tiles."""
    kv = kvattn_lib
    L, n = 900, 300
    mask = seen(range(L - n, L), L, 500, 6)
    c = WindowCache(kv, "bf16", 2, 128, [L], [mask.any(0)], seed=3)
    grow = np.round(1 + np.arange(L) / 150.0)[:, None, None]          # whole numbers 1 .. 7: products with bf16 k
    k = torch.from_numpy(c.k[0] * grow).to(torch.bfloat16)
    tok = np.nonzero(mask.any(0))[0]
    c.cache.k_pool[torch.from_numpy(c.table[0, tok // 16].astype(np.int64)).cuda(), :,
                   torch.from_numpy(tok % 16).cuda()] = k[tok].cuda()
    q = _q(np.random.default_rng(5), (n, 4, 128), "bf16")
    cfg = kv.make_config(4, 2, 128, kv.BF16)
    out = kv.prefill_window(cfg, c.cache, q.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                            torch.tensor([L - n], dtype=torch.int32).cuda(), c.d_table, n, 500, 6)
    assert kv.get_device_status() == 0
    rows = np.arange(0, n, 3)
    want, mag = attend(q[rows].double().numpy(), k.double().numpy(), c.v[0], mask[rows])
    # scores up to 7 times larger: their sums' errors too, 7 * 2^-12 < 2^-9 on a weight
    bound = (2.0 ** -8 + 2.0 ** -9) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(f64(out)[rows] - want) <= bound)


def test_step_of_a_windowed_layer(kvattn_lib):
    """Prompt chunks, then single tokens, through the append, the chunks' and the tokens' attention together, blocks
    given back as they slide out of the window; against the formula over the whole history."""
    kv = kvattn_lib
    hq, hkv, d, window, sinks, block = 8, 2, 128, 100, 4, 16
    g = np.random.default_rng(12)
    cfg = kv.make_config(hq, hkv, d, kv.BF16)
    form = kv.make_rotary("half", 64, "linear", factor=2.0)
    alloc = kv.BlockAllocator(40)
    cache = kv.Cache(*(torch.full((40, hkv, block, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    table = np.full((2, 64), -1, np.int32)
    have = [0, 0]
    hist = [[np.zeros((0, hkv, d)), np.zeros((0, hkv, d))] for _ in range(2)]

    def step(counts):
        pos, seq = [], []
        for s, n in enumerate(counts):
            need = range((have[s] + block - 1) // block, (have[s] + n + block - 1) // block)
            table[s, list(need)] = alloc.alloc(len(need))
            pos += range(have[s], have[s] + n)
            seq += [s] * n
        T = len(pos)
        qkv = torch.from_numpy(g.standard_normal((T, (hq + 2 * hkv) * d))).to(torch.bfloat16).cuda()
        q, k, v = kv.split_qkv(qkv, hq, hkv, d)
        rot = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
        dt = torch.from_numpy(table).cuda()
        p = torch.tensor(pos, dtype=torch.int32).cuda()
        s = torch.tensor(seq, dtype=torch.int32).cuda()
        kv.rotary_append(cfg, form, cache, q, k, v, p, s, dt, q_out=rot)
        at = (dt.long()[s.long(), p.long() // block], slice(None), p.long() % block)
        for i in range(2):
            mine = torch.tensor([x == i for x in seq])
            for j, pool in enumerate((cache.k_pool, cache.v_pool)):
                hist[i][j] = np.concatenate([hist[i][j], f64(pool[at])[mine.numpy()]])
        if all(n == 1 for n in counts):
            n = torch.tensor([h + 1 for h in have], dtype=torch.int32).cuda()
            out = kv.decode_window(cfg, cache, rot, dt, n, max(have) + 1, window, sinks)
        else:
            cu = torch.cumsum(torch.tensor([0, *counts]), 0).int().cuda()
            out = kv.prefill_window(cfg, cache, rot, cu, torch.tensor(have, dtype=torch.int32).cuda(), dt, max(counts),
                                    window, sinks)
        assert kv.get_device_status() == 0
        got, r = f64(out), f64(rot)
        o = 0
        for i, n in enumerate(counts):
            have[i] += n
            want, mag = attend(r[o:o + n], *hist[i], seen(range(have[i] - n, have[i]), have[i], window, sinks))
            check_attention(got[o:o + n], want, mag, "bf16", f"sequence {i} at {have[i]}")
            o += n
            # blocks that the next token no longer sees
            for c in range(1, max(1, (have[i] + 1 - window) // block)):
                if table[i, c] >= 0:
                    b = table[i, c]
                    alloc.free([b])
                    table[i, c] = -1
                    cache.k_pool[int(b)] = cache.v_pool[int(b)] = float("nan")
    step([150, 33])
    step([40, 100])
    for _ in range(40):
        step([1, 1])
    assert (table >= 0).sum() <= 2 * (1 + 100 // block + 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_captured_calls(kvattn_lib, dtype):
    """Decode and prefill captured once and replayed on new lengths and queries."""
    kv = kvattn_lib
    lens = [600, 350]
    c = WindowCache(kv, dtype, 2, 128, lens, [np.ones(L, bool) for L in lens], seed=4)
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    g = np.random.default_rng(5)
    q = _q(g, (2, 8, 128), "bf16").cuda()
    qc = _q(g, (80, 8, 128), "bf16").cuda()
    n = torch.tensor([100, 350], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 50, 80], dtype=torch.int32).cuda()
    prefix = torch.tensor([400, 0], dtype=torch.int32).cuda()
    f8 = dtype == "fp8"
    dec, pre = (kv.decode_window_fp8, kv.prefill_window_fp8) if f8 else (kv.decode_window, kv.prefill_window)
    ws = [torch.empty(kv.decode_window_workspace_size(cfg, 2, 600, 128, 4), dtype=torch.uint8, device="cuda")]
    wp = {}
    if f8:
        wp = dict(workspace=torch.empty(kv.prefill_window_fp8_workspace_size(cfg, 16, c.table.shape[1], 2, 50, 128, 4),
                                        dtype=torch.uint8, device="cuda"))
    a, b = torch.zeros_like(q), torch.zeros_like(qc)

    def both():
        dec(cfg, c.cache, q, c.d_table, n, 600, 128, 4, out=a, workspace=ws[0])
        pre(cfg, c.cache, qc, cu, prefix, c.d_table, 50, 128, 4, out=b, **wp)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    n.copy_(torch.tensor([599, 17], dtype=torch.int32))
    prefix.copy_(torch.tensor([1, 320], dtype=torch.int32))
    q.copy_(q.flip(0))
    a.zero_()
    b.zero_()
    graph.replay()
    got = a.clone(), b.clone()
    both()
    assert kv.get_device_status() == 0
    assert torch.equal(got[0], a) and torch.equal(got[1], b)
    assert torch.isfinite(a).all() and a.abs().sum() > 0 and b.abs().sum() > 0


def test_python_refusals(kvattn_lib):
    """Arguments that are not what the call takes raise, whichever way they were marshalled, and write nothing."""
    kv = kvattn_lib
    c = WindowCache(kv, "bf16", 2, 128, [40], [np.ones(40, bool)], seed=1)
    c8 = WindowCache(kv, "fp8", 2, 128, [40], [np.ones(40, bool)], seed=1)
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    q = _q(np.random.default_rng(0), (1, 8, 128), "bf16").cuda()
    n = torch.tensor([40], dtype=torch.int32).cuda()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 5.0)
    kv.decode_window(cfg, c.cache, q, c.d_table, n, 40, 16, 2, workspace=ws)
    good = dict(cfg=cfg, cache=c.cache, q=q, block_table=c.d_table, seq_lens=n, max_seq_len=40, window=16, num_sinks=2,
                out=out, workspace=ws)
    for bad, error in ((dict(q=q.float()), TypeError), (dict(q=q.cpu()), ValueError), (dict(q=q[:, :4]), ValueError),
                       (dict(q=q.transpose(1, 2)), ValueError), (dict(seq_lens=n.long()), TypeError),
                       (dict(seq_lens=torch.cat([n, n])), ValueError), (dict(block_table=c.d_table[:0]), ValueError),
                       (dict(block_table=c.d_table.cpu()), ValueError), (dict(out=out[:, :4]), ValueError),
                       (dict(out=out.float()), TypeError), (dict(cache=c8.cache), TypeError),
                       (dict(cfg=kv.make_config(8, 4, 128, kv.BF16)), ValueError),
                       (dict(cfg=kv.make_config(8, 2, 128, kv.F32)), TypeError), (dict(window=0), kv.KvattnError),
                       (dict(num_sinks=-1), kv.KvattnError), (dict(workspace=ws[:16], num_splits=4), kv.KvattnError)):
        with pytest.raises(error):
            kv.decode_window(**{**good, **bad})
    qc = q.expand(3, 8, 128).contiguous()
    outc = torch.full_like(qc, 5.0)
    cu = torch.tensor([0, 3], dtype=torch.int32).cuda()
    pre = dict(cfg=cfg, cache=c.cache, q=qc, cu_q_lens=cu, prefix_lens=n - 3, block_table=c.d_table, max_q_len=3, window=16,
               num_sinks=2, out=outc)
    for bad, error in ((dict(q=qc.float()), TypeError), (dict(cu_q_lens=cu[:1]), ValueError),
                       (dict(prefix_lens=(n - 3).long()), TypeError), (dict(out=outc[:2]), ValueError),
                       (dict(block_table=c.d_table[:0]), ValueError), (dict(window=-3), kv.KvattnError)):
        with pytest.raises(error):
            kv.prefill_window(**{**pre, **bad})
    with pytest.raises(kv.KvattnError):
        kv.prefill_window_fp8(**{**pre, "cache": c8.cache}, workspace=ws[:64])
    k = _q(np.random.default_rng(1), (3, 2, 128), "bf16").cuda()
    ints = torch.tensor([1, 2, 3], dtype=torch.int32).cuda()
    app = dict(cfg=cfg, rotary=kv.make_rotary("half"), cache=c.cache, q=qc, k=k, v=k, positions=ints, seq_ids=ints * 0,
               block_table=c.d_table, q_out=outc)
    before = c.cache.k_pool.clone()
    for bad, error in ((dict(q=qc[:2]), ValueError), (dict(k=k.float()), TypeError), (dict(v=k[:, :1]), ValueError),
                       (dict(positions=ints[:2]), ValueError), (dict(seq_ids=ints.long()), TypeError),
                       (dict(q_out=outc[:2]), ValueError), (dict(q=qc.cpu()), ValueError), (dict(cache=c8.cache), TypeError),
                       (dict(rotary=kv.make_rotary("half", 24)), kv.KvattnError)):
        with pytest.raises(error):
            kv.rotary_append(**{**app, **bad})
    torch.cuda.synchronize()
    assert torch.all(out == 5.0) and torch.all(outc == 5.0)
    assert torch.equal(torch.nan_to_num(c.cache.k_pool), torch.nan_to_num(before))
    assert kv.get_device_status() == 0
    kv.decode_window(**good)
    assert torch.all(out != 5.0)


def test_prefill_many_chunks(kvattn_lib):
    """More (chunk, token block) pairs than are ranked in shared memory: 700 chunks of 0 to 3 rows and a long one."""
    g = np.random.default_rng(31)
    chunks = [(int(g.integers(0, 90)), int(g.integers(0, 4))) for _ in range(699)] + [(40, 300)]
    _prefill(kvattn_lib, "bf16", 2, 1, 128, chunks, 33, 2, step=29, seed=7, spare_rows=2)


def test_prefill_long_chunk_among_short(kvattn_lib):
    """A long chunk and many of one row: far fewer token blocks than chunks times the longest chunk's."""
    g = np.random.default_rng(32)
    chunks = [(int(g.integers(0, 60)), 1) for _ in range(150)]
    chunks[70] = (30, 1100)
    _prefill(kvattn_lib, "bf16", 4, 2, 128, chunks, 40, 3, step=97, seed=8)


def test_prefill_thousands_of_chunks(kvattn_lib):
    """More chunks than one launch takes, every one with its own prefix, in two shapes: most of them empty, and none."""
    for least in (0, 1):
        g = np.random.default_rng(33 + least)
        chunks = [(int(g.integers(0, 20)), int(g.integers(least, 2)) if i % 1000 else 9) for i in range(4200)]
        _prefill(kvattn_lib, "bf16", 2, 1, 64, chunks, 11, 2, step=3, seed=9 + least)
    _prefill(kvattn_lib, "fp8", 4, 1, 128, [(i % 37, 1) for i in range(2100)], 11, 2, seed=11)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift", [8, 16])
def test_prefill_out_alignment(kvattn_lib, d, shift):
    """An output on 16 bytes, and on 32: the same values."""
    kv = kvattn_lib
    n = 140
    c = WindowCache(kv, "bf16", 2, d, [n], [np.ones(n, bool)], seed=4)
    cfg = kv.make_config(8, 2, d, kv.BF16)
    q = _q(np.random.default_rng(6), (n, 8, d), "bf16").cuda()
    cu, prefix = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    want = kv.prefill_window(cfg, c.cache, q, cu, prefix, c.d_table, n, 50, 2)
    room = torch.full((q.numel() + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = room[shift:shift + q.numel()].view(q.shape)
    kv.prefill_window(cfg, c.cache, q, cu, prefix, c.d_table, n, 50, 2, out=out)
    assert torch.equal(out, want)
    assert torch.all(room[:shift] == 9.0) and torch.all(room[shift + q.numel():] == 9.0)


def test_prefill_bad_chunks(kvattn_lib):
    """Chunks whose metadata is out of range are skipped and recorded; the others are as without them."""
    kv = kvattn_lib
    chunks = [(100, 30), (50, 40), (0, 20)]
    lens = [p + n for p, n in chunks]
    masks = [seen(range(p, p + n), p + n, 64, 3) for p, n in chunks]
    c = WindowCache(kv, "bf16", 2, 128, lens, [m.any(0) for m in masks], seed=2)
    q = _q(np.random.default_rng(3), (90, 8, 128), "bf16")
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    cu = torch.tensor([0, 30, 70, 90], dtype=torch.int32).cuda()
    for prefix, max_q in (([100, -1, 0], 40), ([100, 10 ** 6, 0], 40), ([100, 50, 0], 39)):
        out = torch.full((90, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        kv.prefill_window(cfg, c.cache, q.cuda(), cu, torch.tensor(prefix, dtype=torch.int32).cuda(), c.d_table, max_q, 64,
                          3, out=out)
        assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
        got = f64(out)
        assert np.all(got[30:70] == 9.0)
        for i, (a, b) in ((0, (0, 30)), (2, (70, 90))):
            want, mag = attend(q[a:b].double().numpy(), c.k[i], c.v[i], masks[i])
            check_attention(got[a:b], want, mag, "bf16", f"chunk {i}")


def test_streams(kvattn_lib):
    """The stream argument, and the current stream, with buffers of another one."""
    kv = kvattn_lib
    c = WindowCache(kv, "bf16", 2, 128, [500], [np.ones(500, bool)], seed=4)
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    q = _q(np.random.default_rng(5), (1, 8, 128), "bf16").cuda()
    qc = q.expand(7, 8, 128).contiguous()
    n = torch.tensor([500], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 7], dtype=torch.int32).cuda()
    want = kv.decode_window(cfg, c.cache, q, c.d_table, n, 500, 99, 4)
    want_c = kv.prefill_window(cfg, c.cache, qc, cu, n - 7, c.d_table, 7, 99, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = kv.decode_window(cfg, c.cache, q, c.d_table, n, 500, 99, 4, stream=side)
    b = kv.prefill_window(cfg, c.cache, qc, cu, n - 7, c.d_table, 7, 99, 4, stream=side)
    with torch.cuda.stream(side):
        a2 = kv.decode_window(cfg, c.cache, q, c.d_table, n, 500, 99, 4, out=torch.empty_like(q),
                              workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(a2, want) and torch.equal(b, want_c)


def test_stream_allocations(kvattn_lib):
    """What a call on a side stream allocates for itself is not given to the current stream while the call waits."""
    kv = kvattn_lib
    c = WindowCache(kv, "fp8", 2, 128, [500], [np.ones(500, bool)], seed=4)
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    q = _q(np.random.default_rng(5), (60, 8, 128), "bf16").cuda()
    cu, prefix = torch.tensor([0, 60], dtype=torch.int32).cuda(), torch.tensor([440], dtype=torch.int32).cuda()
    call = lambda stream: kv.prefill_window_fp8(cfg, c.cache, q, cu, prefix, c.d_table, 60, 99, 4, stream=stream)
    want = call(None)
    size = kv.prefill_window_fp8_workspace_size(cfg, 16, c.d_table.shape[1], 1, 60, 99, 4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    got = call(side)
    for n in (size, q.numel() * 2):
        torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,hkv,d", [("bf16", 8, 128), ("bf16", 8, 64), ("f32", 4, 128)])
def test_far_into_a_large_pool(kvattn_lib, dtype, hkv, d):
    """Blocks whose element offsets pass 2^31 (bytes 2^32), written by the append and read by both attentions."""
    kv = kvattn_lib
    t = TORCH_DT[dtype]
    per = hkv * 16 * d
    blocks = (2 ** 31 + 2 ** 28) // per
    hq = 4 * hkv
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    cache = kv.Cache(*(torch.empty((blocks, hkv, 16, d), dtype=t, device="cuda") for _ in range(2)))
    L = 50
    table = torch.tensor([[0, blocks - 1, blocks - 3, 2 ** 31 // per + 1]], dtype=torch.int32).cuda()
    for b in table[0].tolist():
        cache.k_pool[b] = cache.v_pool[b] = float("nan")
    g = np.random.default_rng(6)
    qkv = torch.from_numpy(g.standard_normal((L, (hq + 2 * hkv) * d))).to(t).cuda()
    q, k, v = kv.split_qkv(qkv, hq, hkv, d)
    rot = torch.empty((L, hq, d), dtype=t, device="cuda")
    pos = torch.arange(L, dtype=torch.int32).cuda()
    kv.rotary_append(cfg, kv.make_rotary("half"), cache, q, k, v, pos, pos * 0, table, q_out=rot)
    from _window_support import rotate, speeds
    keys, _ = rotate(f64(k), np.arange(L), speeds(10000.0, d), d, "half", 1.0)
    keys = torch.from_numpy(keys).to(t).double().numpy()
    stored = f64(cache.k_pool[table[0].long()[pos.long() // 16], :, pos.long() % 16])
    assert np.abs(stored - keys).max() <= 2.0 ** (-6 if dtype == "bf16" else -20)   # a step of values below 8
    mask = seen(range(L), L, 20, 5)
    n = torch.tensor([L], dtype=torch.int32).cuda()
    out = kv.decode_window(cfg, cache, rot[-1:].contiguous(), table, n, L, 20, 5)
    want, mag = attend(f64(rot[-1:]), stored, f64(v), mask[-1:])
    check_attention(f64(out), want, mag, dtype, "decode")
    flat = kv.decode_window(cfg, cache, rot[-1:].contiguous(), table, n, L, 20, 5, num_splits=2)
    check_attention(f64(flat), want, mag, dtype, "decode, split")
    if dtype == "bf16" and blocks * hkv * 16 < 2 ** 31:
        out = kv.prefill_window(cfg, cache, rot, torch.tensor([0, L], dtype=torch.int32).cuda(), n * 0, table, L, 20, 5)
        want, mag = attend(f64(rot), stored, f64(v), mask)
        check_attention(f64(out), want, mag, dtype, "prefill")
    assert kv.get_device_status() == 0


def test_first_call_in_a_capture(kvattn_lib):
    """A process whose first calls are captured: what they set up (attributes, tensor maps) is no stream work."""
    import subprocess
    import sys

    code = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch, kv_cache_attention_rope_gb300 as kv
cfg = kv.make_config(8, 2, 128, kv.BF16)
cache = kv.Cache(*(torch.randn((4, 2, 16, 128), device='cuda').to(torch.bfloat16) for _ in range(2)))
q = torch.randn((3, 8, 128), device='cuda').to(torch.bfloat16)
k = torch.randn((3, 2, 128), device='cuda').to(torch.bfloat16)
table = torch.arange(4, dtype=torch.int32, device='cuda')[None]
pos = torch.tensor([20, 21, 22], dtype=torch.int32, device='cuda')
ids, n = pos * 0, torch.tensor([23], dtype=torch.int32, device='cuda')
cu, prefix = torch.tensor([0, 3], dtype=torch.int32, device='cuda'), torch.tensor([20], dtype=torch.int32, device='cuda')
rot, a, b = torch.empty_like(q), torch.zeros_like(q[:1]), torch.zeros_like(q)
ws = torch.empty(1 << 20, dtype=torch.uint8, device='cuda')
def calls():
    kv.rotary_append(cfg, kv.make_rotary('half'), cache, q, k, k, pos, ids, table, q_out=rot)
    kv.decode_window(cfg, cache, rot[2:], table, n, 64, 16, 2, out=a, workspace=ws)
    kv.decode_window(cfg, cache, rot[2:], table, n, 64, 16, 2, out=a, workspace=ws, num_splits=2)
    kv.prefill_window(cfg, cache, rot, cu, prefix, table, 3, 16, 2, out=b)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = a.clone(), b.clone()
calls()
torch.cuda.synchronize()
assert kv.get_device_status() == 0 and torch.equal(got[0], a) and torch.equal(got[1], b) and a.abs().sum() > 0
print('captured')
"""
    import os

    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code % (os.path.dirname(here), here)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr
