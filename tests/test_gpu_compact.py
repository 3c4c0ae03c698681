"""GPU tests of token compaction and of block copies in an fp8 cache: bit copies, every other slot as it was."""
import numpy as np
import pytest
import torch

from _shared_support import compacted, compacted_pages

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 1), ("f32", 1), ("fp8", 1), ("bf16", 3), ("f32", 2)]


class Case:
    """Sequences in a pool of random bits, and what they keep."""

    def __init__(self, kv, dtype, layers, hkv, d, lens, starts, lists, block=16, seed=0):
        g = np.random.default_rng(seed)
        self.kv, self.dtype, self.layers, self.block = kv, dtype, layers, block
        need = [(n + block - 1) // block for n in lens]
        self.nb = sum(need) + 2
        ids = g.permutation(self.nb)
        self.table = np.full((len(lens), max(need)), -1, np.int32)
        o = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[o:o + n]
            o += n
        self.starts, self.lists = list(starts), [list(k) for k in lists]
        if dtype == "fp8":
            self.raw = torch.from_numpy(g.integers(0, 256, (self.nb, hkv, block // 16, 4224), dtype=np.uint8)).cuda()
            self.cache = kv.CacheFP8(self.raw, block)
        else:
            t, bits = (torch.bfloat16, np.int16) if dtype == "bf16" else (torch.float32, np.int32)
            shape = (layers, 2, self.nb, hkv, block, d)
            x = g.integers(np.iinfo(bits).min, np.iinfo(bits).max, shape, dtype=bits)
            self.raw = torch.from_numpy(x).cuda()
            pool = self.raw.view(t)
            cfg = kv.make_config(hkv, hkv, d, kv.BF16 if dtype == "bf16" else kv.F32)
            self.cache = kv.LayeredCache(cfg, pool) if layers > 1 else kv.Cache(pool[0, 0], pool[0, 1])
        self.cfg = kv.make_config(hkv, hkv, d, kv.F32 if dtype == "f32" else kv.BF16)
        self.before = self.raw.cpu().numpy().copy()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.ints = [torch.from_numpy(self.table).cuda(), i32(self.starts),
                     i32(np.cumsum([0] + [len(k) for k in self.lists]).tolist()), i32([p for k in self.lists for p in k])]

    def want(self, before=None):
        f = compacted_pages if self.dtype == "fp8" else compacted
        return f(self.before if before is None else before, self.table, self.starts, self.lists, self.block)

    def run(self, **more):
        self.kv.compact_tokens(self.cfg, self.cache, *self.ints, **more)

    def check(self, want=None):
        assert self.kv.get_device_status() == 0
        assert np.array_equal(self.raw.cpu().numpy(), self.want() if want is None else want)


def _some(g, start, stop, share):
    return [p for p in range(start, stop) if g.random() < share]


@pytest.mark.parametrize("dtype,layers", KINDS)
@pytest.mark.parametrize("hkv,d,block", [(8, 128, 16), (12, 64, 16), (1, 128, 48), (3, 64, 32)])
def test_ragged(kvattn_lib, dtype, layers, hkv, d, block):
    """Nothing kept, everything kept, one token, tokens that stay, drafts at the end, long lists."""
    g = np.random.default_rng(hkv + d)
    d = 128 if dtype == "fp8" else d
    lens = [40, 33, 1, 17, 100, 300, 64, 1500, 700, 16]
    starts = [0, 0, 0, 16, 76, 5, 0, 0, 699, 15]
    lists = [[], range(33), [0], [16], [77, 80, 99], _some(g, 5, 300, 0.5), range(32, 64), _some(g, 0, 1500, 0.7), [699],
             [15]]
    c = Case(kvattn_lib, dtype, layers, hkv, d, lens, starts, lists, block=block, seed=d)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,layers", KINDS)
@pytest.mark.parametrize("share", [0.05, 0.5, 0.95])
@pytest.mark.parametrize("start", [0, 7, 16, 100])
def test_shares(kvattn_lib, dtype, layers, share, start):
    g = np.random.default_rng(int(100 * share) + start)
    c = Case(kvattn_lib, dtype, layers, 2, 128, [2000, 333], [start, start],
             [_some(g, start, 2000, share), _some(g, start, 333, share)], seed=start)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,layers", KINDS)
def test_shifts(kvattn_lib, dtype, layers):
    """Every token one, fifteen, sixteen, seventeen places down: each round reads what the next one's places were."""
    shifts = [1, 15, 16, 17, 31, 64, 129, 1000]
    c = Case(kvattn_lib, dtype, layers, 4, 128, [2100] * len(shifts), [0] * len(shifts),
             [range(s, 2100) for s in shifts], seed=1)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,layers", KINDS)
def test_many_sequences(kvattn_lib, dtype, layers):
    """Drafts of many sequences: a few tokens each."""
    g = np.random.default_rng(2)
    lens = [int(n) + 24 for n in g.integers(1, 200, 150)]
    lists = [[n - 24] + _some(g, n - 23, n, 0.2) for n in lens]
    c = Case(kvattn_lib, dtype, layers, 8, 128, lens, [n - 24 for n in lens], lists, seed=2)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,layers", KINDS)
def test_one_long_sequence(kvattn_lib, dtype, layers):
    g = np.random.default_rng(3)
    c = Case(kvattn_lib, dtype, layers, 1, 128, [40000], [3], [_some(g, 3, 40000, 0.5)], seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,layers", KINDS)
def test_twice_on_a_stream_and_captured(kvattn_lib, dtype, layers):
    kv = kvattn_lib
    g = np.random.default_rng(4)
    c = Case(kv, dtype, layers, 2, 128, [500, 90], [0, 20], [_some(g, 0, 500, 0.8), _some(g, 20, 90, 0.8)], seed=4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    graph.replay()
    once = c.want()
    c.check(once)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)  # over what the first left
    torch.cuda.current_stream().wait_stream(side)
    c.check(c.want(once))


@pytest.mark.parametrize("dtype,layers", [("bf16", 1), ("fp8", 1), ("bf16", 2)])
def test_bad_lists(kvattn_lib, dtype, layers):
    """Lists that do not ascend, lie before their places or outside `keep`, places and blocks that are not there: reported,
    with every other sequence as it should be and nothing written outside the sequence's own blocks."""
    kv = kvattn_lib
    bad = kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    lens, starts = [100, 100, 100], [0, 10, 0]
    lists = [[3, 5, 50, 99], [12, 30, 31, 32, 90], [1, 2, 64]]

    def run(change, same=(0, 2)):
        c = Case(kv, dtype, layers, 2, 128, lens, starts, lists, seed=5)
        change(*c.ints)
        c.run()
        assert kv.get_device_status() == bad
        got, want = c.raw.cpu().numpy(), c.want()
        axis = 0 if dtype == "fp8" else 2
        own = {int(b) for b in c.table[1] if b >= 0}
        for b in range(c.nb):
            if b not in own:
                assert np.array_equal(np.take(got, b, axis), np.take(want, b, axis))
        return c, got

    def set_(i, at, value):
        def f(*ints):
            ints[i][at] = value
        return f

    run(set_(3, 6, 12))             # not ascending
    run(set_(3, 6, 10))             # before its place
    run(set_(3, 6, -5))
    run(set_(3, 8, 2 ** 31 - 1))    # outside the table
    run(set_(1, 1, 2 ** 31 - 3))    # places outside the table
    run(set_(1, 1, -1))
    c, got = run(set_(0, (1, 5), -1))         # the block of position 90
    c, got = run(set_(0, (1, 1), 2 ** 31 - 1))
    # lists that overlap or lie outside keep: each counts as empty
    c = Case(kv, dtype, layers, 2, 128, lens, starts, lists, seed=6)
    c.ints[2].copy_(torch.tensor([0, 40, -1, 12], dtype=torch.int32))
    c.run()
    assert kv.get_device_status() == bad
    assert np.array_equal(c.raw.cpu().numpy(), c.before)


def test_bad_lists_move_the_good_tokens(kvattn_lib):
    """A kept token whose block is not there stays; the list's others move."""
    kv = kvattn_lib
    c = Case(kv, "bf16", 1, 2, 128, [100], [10], [[12, 30, 31, 32, 90]], seed=7)
    c.ints[0][0, 5] = -1
    c.run()
    assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]
    c.lists = [[12, 30, 31, 32]]
    assert np.array_equal(c.raw.cpu().numpy(), c.want())


def test_offsets_past_32_bits(kvattn_lib):
    """A pool of more than 2^32 bytes, its first and last blocks."""
    kv = kvattn_lib
    nb = 140000
    pool = torch.zeros((2, nb, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    cache = kv.Cache(pool[0], pool[1])
    cfg = kv.make_config(8, 8, 128, kv.BF16)
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = [nb - 1, 0, nb - 2]
    for b in ids:
        pool[:, b] = torch.randn(pool[:, b].shape, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    before = pool[:, ids].clone()
    keep = [5, 17, 18, 40]
    kv.compact_tokens(cfg, cache, i32(ids), i32(0), i32(0, 4), i32(*keep))
    assert kv.get_device_status() == 0
    line = before.permute(0, 1, 3, 2, 4).reshape(2, 48, 8, 128)
    line[:, :4] = line[:, keep].clone()
    assert torch.equal(pool[:, ids], line.view(2, 3, 16, 8, 128).permute(0, 1, 3, 2, 4))
    del pool, cache
    pages = torch.zeros((nb, 8, 1, 4224), dtype=torch.uint8, device="cuda")
    cache = kv.CacheFP8(pages)
    pages[nb - 1] = torch.randint(0, 256, pages[0].shape, dtype=torch.uint8, device="cuda")
    kv.copy_blocks(cfg, cache, [nb - 1], [nb - 2])
    assert kv.get_device_status() == 0
    assert torch.equal(pages[nb - 1], pages[nb - 2]) and not pages[nb - 3].any()


@pytest.mark.parametrize("n", [1, 3, 64, 500])
@pytest.mark.parametrize("hkv,block", [(8, 16), (1, 16), (3, 48), (32, 16)])
def test_copy_blocks_fp8(kvattn_lib, n, hkv, block):
    kv = kvattn_lib
    g = np.random.default_rng(n)
    nb = 2 * n + 3
    pages = torch.from_numpy(g.integers(0, 256, (nb, hkv, block // 16, 4224), dtype=np.uint8)).cuda()
    cache, cfg = kv.CacheFP8(pages, block), kv.make_config(hkv, hkv, 128, kv.BF16)
    ids = g.permutation(nb)
    src, dst = ids[:n].tolist(), ids[n:2 * n].tolist()
    src[-1] = src[0]  # one source twice
    want = pages.clone()
    want[dst] = pages[src]
    kv.copy_blocks(cfg, cache, src, dst)
    assert kv.get_device_status() == 0 and torch.equal(pages, want)
    # pairs with an id outside the pool are skipped and reported
    bad = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (src, dst)]
    bad[0][0], bad[1][n // 2] = -1, nb
    pages.copy_(torch.from_numpy(g.integers(0, 256, pages.shape, dtype=np.uint8)))
    want = pages.clone()
    for s, d in zip(*(b.tolist() for b in bad)):
        if s >= 0 and d < nb:
            want[d] = pages[s]
    kv.copy_blocks(cfg, cache, *bad)
    assert kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"] and torch.equal(pages, want)
    kv.copy_blocks(cfg, cache, [], [])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv.copy_blocks(cfg, cache, *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (src, dst)), stream=side)
    torch.cuda.synchronize()
    assert kv.get_device_status() == 0


def test_refusals_of_tensors(kvattn_lib):
    kv = kvattn_lib
    c = Case(kv, "bf16", 1, 2, 128, [40], [0], [[3, 5]])
    table, starts, cu, keep = c.ints
    for wrong in ((table.long(), starts, cu, keep), (table, starts[:0], cu, keep), (table, starts, cu[:1], keep),
                  (table, starts, cu, keep.cpu()), (table, starts, cu, keep.float()), (table[:0], starts, cu, keep),
                  (table, starts, cu, keep.view(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            kv.compact_tokens(c.cfg, c.cache, *wrong)
    with pytest.raises((TypeError, ValueError)):
        kv.compact_tokens(kv.make_config(4, 4, 128, kv.BF16), c.cache, *c.ints)
    with pytest.raises((TypeError, ValueError)):
        kv.compact_tokens(kv.make_config(2, 2, 128, kv.F32), c.cache, *c.ints)
    assert np.array_equal(c.raw.cpu().numpy(), c.before)
