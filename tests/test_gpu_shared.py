"""GPU tests of decode over shared prefixes against the formula in 64 bits, every sequence by itself.

Slots that no sequence sees hold NaN and table entries without a seen token are -1.  Tolerances:
_window_support.check_attention, for fp8 pages as for bf16 (over a prefix a weight times its V scale is rounded to bf16,
2^-8; codes and scores are exact or fp32); the merge of the two parts of a sequence is in fp32 and adds less than the
exp2 that it counts.
"""
import numpy as np
import pytest
import torch

from _shared_support import SharedCache
from _window_support import TORCH_DT, attend, check_attention
from _gpu_support import f64

pytestmark = pytest.mark.gpu

# A bound of the shared lengths by which a small call counts as one that gains from reading prefixes once.
LOOSE = 1 << 20


def _want(c, q):
    return [attend(q[r:r + 1], c.k[r], c.v[r], np.ones((1, n), bool)) for r, n in enumerate(c.lens)]


def _check(c, q, got, dtype, what=""):
    for r, (want, mag) in enumerate(_want(c, q.double().cpu().numpy())):
        check_attention(got[r:r + 1], want, mag, "f32" if dtype == "f32" else "bf16", f"{what} sequence {r} of length {c.lens[r]}")
        if c.lens[r] == 0:
            assert np.all(got[r] == 0.0)


def _q(g, shape, dtype):
    return torch.from_numpy(g.standard_normal(shape)).to(TORCH_DT["f32" if dtype == "f32" else "bf16"])


def _run(kv, dtype, hq, hkv, d, groups, block=16, seed=0, **more):
    c = SharedCache(kv, dtype, hkv, d, groups, block=block, seed=seed, **more)
    q = _q(np.random.default_rng(seed + 1), (len(c.lens), hq, d), dtype)
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    for most in (int(c.shared.max()), LOOSE):  # each sequence by itself where the call is small, prefixes once
        out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
        size = kv.decode_shared_workspace_size(cfg, len(c.lens), max(max(c.lens), 1), len(c.shared), most)
        workspace = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN to whoever reads it first
        call(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, max(max(c.lens), 1), c.d_cu, c.d_shared, most, out=out,
             workspace=workspace)
        assert kv.get_device_status() == 0
        _check(c, q, f64(out), dtype, f"bound {most}")
    return c, q, cfg, out


HEADS = [("bf16", 32, 8, 128), ("bf16", 64, 8, 128), ("bf16", 4, 4, 128), ("bf16", 4, 2, 128), ("bf16", 12, 12, 64),
         ("bf16", 8, 1, 64), ("bf16", 4, 1, 64), ("bf16", 4, 2, 64), ("f32", 12, 12, 64), ("f32", 8, 2, 128),
         ("fp8", 8, 2, 128), ("fp8", 16, 2, 128)]
FP8_GROUPS = (4, 8)


@pytest.mark.parametrize("dtype,hq,hkv,d", HEADS)
@pytest.mark.parametrize("groups", [
    [(100, [101, 130, 100, 164])],
    [(512, [513] * 5 + [600])],
    [(1000, [1000 + 7 * i for i in range(40)])],
    # several groups: single sequences, short and unaligned prefixes, empty places, sequences that end inside the prefix
    [(0, [5, 0]), (33, [34, 0, 60, 33]), (700, [0, 0]), (16, [17, 40]), (1024, [1500, 1024, 1100, 40, 0, 1023, 1029]),
     (300, [301]), (15, [16, 15])],
])
def test_groups(kvattn_lib, dtype, hq, hkv, d, groups):
    _run(kvattn_lib, dtype, hq, hkv, d, groups, seed=hq + d + len(groups))


@pytest.mark.parametrize("shared", [127, 128, 129, 143, 144, 255, 256, 257, 1024, 2047])
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("fp8", 8, 2, 128)])
def test_prefix_lengths(kvattn_lib, dtype, hq, hkv, d, shared):
    _run(kvattn_lib, dtype, hq, hkv, d, [(shared, [shared + 1, shared, shared + 50, shared + 17])], seed=shared)


@pytest.mark.parametrize("n", [2, 3, 31, 32, 33, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 2, 2, 64), ("fp8", 8, 1, 128)])
def test_sequences_of_a_group(kvattn_lib, dtype, hq, hkv, d, n):
    """Groups that fill the rows of a tile, and one more or fewer."""
    _run(kvattn_lib, dtype, hq, hkv, d, [(400, [401 + i % 40 for i in range(n)])], seed=n)


@pytest.mark.parametrize("dtype,hq,hkv,d,block", [("bf16", 8, 2, 128, 32), ("bf16", 8, 2, 128, 128), ("bf16", 4, 4, 64, 48),
                                                  ("fp8", 8, 2, 128, 32), ("f32", 4, 2, 64, 32)])
def test_block_sizes(kvattn_lib, dtype, hq, hkv, d, block):
    _run(kvattn_lib, dtype, hq, hkv, d, [(500, [520, 501, 700]), (90, [91, 300])], block=block, seed=block)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("f32", 12, 12, 64), ("bf16", 4, 4, 64)])
@pytest.mark.parametrize("block", [784, 777])
def test_contiguous_cache(kvattn_lib, dtype, hq, hkv, d, block):
    """One row per sequence, the common tokens in each; of a length that is no multiple of 16 too."""
    _run(kvattn_lib, dtype, hq, hkv, d, [(600, [601, 777, 0, 650])], block=block, own_rows=True, seed=block)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 12, 12, 64), ("fp8", 32, 8, 128)])
def test_long_prefix(kvattn_lib, dtype, hq, hkv, d):
    """Many key ranges of one prefix."""
    _run(kvattn_lib, dtype, hq, hkv, d, [(9000, [9001, 9300, 9017])], seed=3)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 16, 4, 128), ("bf16", 4, 4, 64), ("bf16", 8, 1, 64), ("fp8", 8, 1, 128),
                                            ("bf16", 2, 1, 128)])
@pytest.mark.parametrize("groups", [
    [(300, [301, 5000, 310, 4396, 4397]), (0, [4500])],
    [(5000, [5001, 5100, 9200, 0]), (64, [4160, 4161, 4159, 70])],
    [(16, [5000, 17, 16])],
])
def test_long_own_parts(kvattn_lib, dtype, hq, hkv, d, groups):
    """Sequences with many keys of their own, cut into many pieces, beside ones with few."""
    _run(kvattn_lib, dtype, hq, hkv, d, groups, seed=hkv)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("fp8", 8, 2, 128), ("f32", 4, 2, 64)])
def test_growing_scores(kvattn_lib, dtype, hq, hkv, d):
    """Keys that grow along the sequence: the maximum rises tile by tile, and lies in the prefix or in the own tokens."""
    kv = kvattn_lib
    c = SharedCache(kv, dtype, hkv, d, [(640, [641, 700, 640])], seed=5)
    q = _q(np.random.default_rng(6), (3, hq, d), dtype)
    scale = np.linspace(0.1, 4.0, 700)
    if dtype == "fp8":
        s = c.cache.pool.view(torch.float32)
        for r, n in enumerate(c.lens):
            for p in range(0 if r == 0 else 640, n):
                b = int(c.table[r, p // 16])
                s[b, :, 0, 1024 + p % 16] *= scale[p]
    else:
        for r, n in enumerate(c.lens):
            for p in range(0 if r == 0 else 640, n):
                c.cache.k_pool[int(c.table[r, p // 16]), :, p % 16] *= scale[p]
    for r, n in enumerate(c.lens):  # what is held now
        at = torch.from_numpy(c.table[r, np.arange(n) // 16].astype(np.int64)).cuda(), torch.arange(n).cuda() % 16
        if dtype == "fp8":
            ratio = np.float32(scale[:n])
            c.k[r] = np.float64(np.float32(1) * c.k[r]) * ratio[:, None, None]
        else:
            c.k[r] = f64(c.cache.k_pool[at[0], :, at[1]])
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    got = f64(call(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, 700, c.d_cu, c.d_shared, LOOSE))
    assert kv.get_device_status() == 0
    for r, (want, mag) in enumerate(_want(c, q.double().numpy())):
        if dtype == "f32":  # the scores reach 16: their fp32 sums are off by 2^-12 absolute at most
            assert np.all(np.abs(got[r] - want[0]) <= 2.0 ** -11 * mag[0] + 2.0 ** -23 * np.abs(want[0]))
            continue
        # as check_attention, with scores up to 16 times larger, and so their fp32 sums' errors; fp8's scales are
        # rounded once more by the test's product (2^-24)
        weight = 2.0 ** -8 + 2.0 ** -9
        bound = weight * mag[0] + 2.0 ** -8 * (np.abs(want[0]) + weight * mag[0])
        assert np.all(np.abs(got[r] - want[0]) <= bound), r


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("fp8", 8, 2, 128), ("f32", 4, 2, 64)])
def test_nan_stays_with_its_sequence(kvattn_lib, dtype, hq, hkv, d):
    """A NaN in one sequence's own tokens, or its query, leaves the others' results as they were; one in the prefix is
    everyone's who has it."""
    kv = kvattn_lib
    groups = [(300, [301, 340, 0, 17, 330])]
    c, q, cfg, out = _run(kv, dtype, hq, hkv, d, groups, seed=8)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    args = (c.d_table, c.d_lens, 340, c.d_cu, c.d_shared, LOOSE)
    q2 = q.cuda()
    q2[4] = float("nan")
    got = call(cfg, c.cache, q2, *args)
    assert torch.isnan(got[4]).all() and torch.equal(got[:4], out[:4])
    b, r = int(c.table[1, 320 // 16]), 320 % 16
    if dtype == "fp8":
        c.cache.pool[b, :, 0, r * 128:(r + 1) * 128] = 0x7F
    else:
        c.cache.k_pool[b, :, r] = float("nan")
    got = call(cfg, c.cache, q.cuda(), *args)
    assert torch.isnan(got[1]).all()
    for i in (0, 2, 3, 4):
        assert torch.equal(got[i], out[i])
    b = int(c.table[0, 100 // 16])
    if dtype == "fp8":
        c.cache.pool[b, :, 0, (100 % 16) * 128:(100 % 16 + 1) * 128] = 0x7F
    else:
        c.cache.k_pool[b, :, 100 % 16] = float("nan")
    got = call(cfg, c.cache, q.cuda(), *args)
    for i in (0, 1, 4):
        assert torch.isnan(got[i]).all()
    assert torch.equal(got[2:4], out[2:4])
    assert kv.get_device_status() == 0


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("fp8", 8, 2, 128), ("f32", 4, 2, 64)])
def test_bad_groups_share_nothing(kvattn_lib, dtype, hq, hkv, d):
    """Groups out of order or past the batch, and shared lengths below 0 or above the bound, leave the results as they are
    (and are reported by the calls that look at them); so do sequences past the last group."""
    kv = kvattn_lib
    c, q, cfg, out = _run(kv, dtype, hq, hkv, d, [(260, [261, 300, 290]), (400, [401, 450])], seed=9)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    bad = kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for cu, shared, status in ((i32(0, 3, 6), i32(260, 400), bad), (i32(0, 4, 3), i32(260, 400), bad),
                               (i32(-1, 3, 5), i32(260, 400), bad), (i32(0, 3, 5), i32(260, LOOSE + 1), bad),
                               (i32(0, 3, 5), i32(-1, 400), bad), (i32(0, 3, 3), i32(260, 400), 0),
                               (i32(0), i32(), 0), (i32(0, 0, 3), i32(400, 260), 0), (i32(2, 3, 5), i32(260, 400), bad)):
        got = call(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, 450, cu, shared, LOOSE)
        assert kv.get_device_status() == (0 if dtype == "f32" else status), (cu, shared)
        _check(c, q, f64(got), dtype, str(cu.tolist()))


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("fp8", 8, 2, 128), ("f32", 4, 2, 64)])
def test_bad_lengths_and_blocks(kvattn_lib, dtype, hq, hkv, d):
    """A length above the bound gives zeros; a block outside the pool is reported; the other sequences keep their results."""
    kv = kvattn_lib
    c, q, cfg, out = _run(kv, dtype, hq, hkv, d, [(260, [261, 300, 290, 280])], seed=10)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    bad = kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    for wrong in (301, -1, 2 ** 31 - 1):
        lens = c.d_lens.clone()
        lens[1] = wrong
        got = call(cfg, c.cache, q.cuda(), c.d_table, lens, 300, c.d_cu, c.d_shared, LOOSE)
        assert kv.get_device_status() == bad
        assert torch.all(got[1] == 0)
        _check(SubCase(c, [0, 2, 3]), q[[0, 2, 3]], f64(got[[0, 2, 3]]), dtype)
    for block in (-1, 2 ** 31 - 1, c.cache.num_blocks):
        table = c.d_table.clone()
        table[2, 17] = block  # a block of its own tokens
        got = call(cfg, c.cache, q.cuda(), table, c.d_lens, 300, c.d_cu, c.d_shared, LOOSE)
        assert kv.get_device_status() == bad
        _check(SubCase(c, [0, 1, 3]), q[[0, 1, 3]], f64(got[[0, 1, 3]]), dtype)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 12, 12, 64), ("fp8", 32, 8, 128)])
def test_offsets_past_32_bits(kvattn_lib, dtype, hq, hkv, d):
    """The blocks of a batch at the end of a pool of over 4 GB, the prefix partly there."""
    kv = kvattn_lib
    c = SharedCache(kv, dtype, hkv, d, [(520, [521, 600, 533]), (0, [40])], seed=14)
    small = [c.cache.pool] if dtype == "fp8" else [c.cache.k_pool, c.cache.v_pool]
    count = 2 ** 32 // (small[0][0].numel() * small[0].element_size()) + 200
    pools = [torch.empty((count,) + p.shape[1:], dtype=p.dtype, device="cuda") for p in small]
    n = small[0].shape[0]
    ids = torch.from_numpy(np.where(np.arange(n) % 3 == 0, np.arange(n), count - n + np.arange(n))).cuda()
    for big, p in zip(pools, small):
        big[ids] = p
    c.cache = kv.CacheFP8(*pools) if dtype == "fp8" else kv.Cache(*pools)
    c.d_table = torch.where(c.d_table >= 0, ids[c.d_table.clamp(min=0).long()], -1).int()
    q = _q(np.random.default_rng(15), (len(c.lens), hq, d), dtype)
    cfg = kv.make_config(hq, hkv, d, kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    for most in (520, LOOSE):
        got = call(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, max(c.lens), c.d_cu, c.d_shared, most)
        assert kv.get_device_status() == 0
        _check(c, q, f64(got), dtype, f"bound {most}")


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 4, 1, 64), ("fp8", 4, 1, 128)])
@pytest.mark.parametrize("groups,n", [(192, 2), (193, 2), (1, 2048), (1, 2049), (100, 20)])
def test_many_groups_and_sequences(kvattn_lib, dtype, hq, hkv, d, groups, n):
    """The most groups and sequences whose prefixes are read once, and one more of each."""
    _run(kvattn_lib, dtype, hq, hkv, d, [(128 + 16 * (g % 3), [130 + 16 * (g % 3) + i % 5 for i in range(n)])
                                         for g in range(groups)], seed=16)


class SubCase:
    def __init__(self, c, rows):
        self.k, self.v, self.lens = [c.k[r] for r in rows], [c.v[r] for r in rows], [c.lens[r] for r in rows]


def test_same_as_decode(kvattn_lib):
    """What decode gives over the same tables, up to the roundings of both."""
    kv = kvattn_lib
    c, q, cfg, out = _run(kv, "bf16", 32, 8, 128, [(2000, [2001 + 13 * i for i in range(20)])], seed=11)
    again = kv.decode_shared(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, max(c.lens), c.d_cu, c.d_shared, 2000)
    assert torch.equal(again, out)  # large enough to read the prefix once by its own bound
    other = kv.decode(cfg, c.cache, q.cuda(), c.d_table, c.d_lens, max(c.lens))
    assert float((out.float() - other.float()).abs().max()) < 2e-2


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 12, 12, 64), ("fp8", 32, 8, 128), ("f32", 8, 2, 64)])
def test_streams_and_graphs(kvattn_lib, dtype, hq, hkv, d):
    """On another stream, twice at once with a workspace each, and captured: first call inside the capture, replayed over
    new inputs."""
    kv = kvattn_lib
    c = SharedCache(kv, dtype, hkv, d, [(1030, [1031 + 3 * i for i in range(9)]), (70, [71, 90, 0])], seed=12)
    g = np.random.default_rng(13)
    qs = [_q(g, (len(c.lens), hq, d), dtype).cuda() for _ in range(2)]
    cfg = kv.make_config(hq, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
    call = kv.decode_shared_fp8 if dtype == "fp8" else kv.decode_shared
    args = (c.d_table, c.d_lens, max(c.lens), c.d_cu, c.d_shared, LOOSE)
    size = max(256, kv.decode_shared_workspace_size(cfg, len(c.lens), max(c.lens), 2, LOOSE))
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(qs[0]) for _ in range(2)]
    q = qs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cfg, c.cache, q, *args, out=outs[0], workspace=spaces[0])
    want = [call(cfg, c.cache, x, *args) for x in qs]
    for x, w in zip(qs, want):
        q.copy_(x)
        outs[0].fill_(5.0)
        graph.replay()
        assert torch.equal(outs[0], w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(cfg, c.cache, qs[i], *args, out=outs[i], workspace=spaces[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    got = call(cfg, c.cache, qs[0], *args, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(got, want[0])
    assert kv.get_device_status() == 0


def test_refusals_of_tensors(kvattn_lib):
    kv = kvattn_lib
    c = SharedCache(kv, "bf16", 2, 128, [(32, [33, 40])])
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, block_table=c.d_table, seq_lens=c.d_lens, max_seq_len=40, cu_groups=c.d_cu, shared_lens=c.d_shared,
                max_shared_len=32)
    kv.decode_shared(cfg, c.cache, **good)
    for name, wrong in (("q", q[:, :4]), ("q", q.float()), ("q", q.cpu()), ("seq_lens", c.d_lens.long()),
                        ("seq_lens", c.d_lens[:1]), ("cu_groups", c.d_cu[:1]), ("cu_groups", c.d_cu.cpu()),
                        ("shared_lens", c.d_shared.float()), ("block_table", c.d_table[:1]), ("max_shared_len", 2 ** 31)):
        with pytest.raises((TypeError, ValueError)):
            kv.decode_shared(cfg, c.cache, **{**good, name: wrong})
    with pytest.raises(kv.KvattnError):
        kv.decode_shared(cfg, c.cache, **{**good, "max_shared_len": -1})
    with pytest.raises((TypeError, ValueError)):
        kv.decode_shared_fp8(cfg, c.cache, **good)
