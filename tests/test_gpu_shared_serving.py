"""GPU test of the calls for batches that share prompts, run together as a server would.

Two prompts with images are appended (rotary_append_axes), each is forked to several samples (BlockAllocator.fork,
prepare_append, copy_blocks), the samples grow a token a step and attend (decode_shared), some of their own tokens are
evicted (compact_tokens, BlockAllocator.shrink), and they grow and attend again.  What the cache should hold is followed on
the host: a row is read back once, where it was appended, compared with the rotation in 64 bits, and from then on only
moved in lists; the attention of every step is compared with the formula in 64 bits over these lists.

Tolerances: rows of a bf16 cache as test_gpu_rotary_append; of an fp8 cache half an e4m3 step, 2^-4 of a value or 2^-10
of its row's scale, of what bf16 rounding (2^-8) leaves.  Attention as test_gpu_shared.
"""
import numpy as np
import pytest
import torch

from oracle import fp8
from _gpu_support import f64
from _window_support import attend, check_attention, speeds
from test_gpu_fp8 import unpack_rows
from test_gpu_rotary_append import _close
from test_gpu_rotary_axes import axis_of_pairs, rotate_axes

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCK, WIDTH, NB = 8, 2, 128, 16, 24, 160
SECTIONS, LOOSE = [16, 24, 24], 1 << 20


class Server:
    def __init__(self, kv, kind, rows, seed):
        self.kv, self.fp8 = kv, kind == "fp8"
        self.g = np.random.default_rng(seed)
        self.cfg = kv.make_config(HQ, HKV, D, kv.BF16)
        self.rotary, self.axes = kv.make_rotary("half", 128), kv.make_axes(SECTIONS)
        self.axis = axis_of_pairs(SECTIONS, "sections", 64)
        self.alloc = kv.BlockAllocator(NB)
        self.alloc.alloc(3)  # blocks of others
        if self.fp8:  # NaN codes and scales where nothing was written
            self.cache = kv.CacheFP8(torch.full((NB, HKV, 1, 4224), 0xFF, dtype=torch.uint8, device="cuda"))
        else:
            self.cache = kv.Cache(*(torch.full((NB, HKV, BLOCK, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                                    for _ in range(2)))
        self.table = np.full((rows, WIDTH), -1, np.int32)
        self.k, self.v = [[] for _ in range(rows)], [[] for _ in range(rows)]  # of each sequence's tokens, in 64 bits

    def device(self, x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def append(self, rows, slots, positions):
        """One token per entry: random q, k and v at slots of `rows`, positions [3, T]."""
        T = len(rows)
        x = torch.from_numpy(self.g.standard_normal((T, HQ + 2 * HKV, D))).to(torch.bfloat16)
        dev = x.cuda()
        q, k, v = dev[:, :HQ], dev[:, HQ:HQ + HKV], dev[:, HQ + HKV:]
        q_out = torch.empty((T, HQ, D), dtype=torch.bfloat16, device="cuda")
        call = self.kv.rotary_append_axes_fp8 if self.fp8 else self.kv.rotary_append_axes
        call(self.cfg, self.rotary, self.axes, self.cache, q, k, v, self.device(positions), self.device(slots),
             self.device(rows), torch.from_numpy(self.table).cuda(), q_out=q_out)
        want, size = rotate_axes(x.double().numpy()[:, :HQ + HKV], np.asarray(positions), self.axis, speeds(10000.0, 128), 128,
                                 "half")
        _close(f64(q_out), want[:, :HQ], size[:, :HQ], "bf16", "q")
        blk, off = self.table[rows, np.asarray(slots) // BLOCK], np.asarray(slots) % BLOCK
        wk, wv = want[:, HQ:], x.double().numpy()[:, HQ + HKV:]
        if self.fp8:
            ck, sk, cv, sv = unpack_rows(self.cache.pool.cpu().numpy(), blk, off)
            got = fp8.dequantize_rows(ck, sk), fp8.dequantize_rows(cv, sv)
            for have, exact, more in ((got[0], wk, size[:, HQ:]), (got[1], wv, 0.0)):
                scale = np.abs(exact).max(-1, keepdims=True) / 448 * (1 + 2.0 ** -7)
                bound = (2.0 ** -4 * (1 + 2.0 ** -8) + 2.0 ** -8) * np.abs(exact) + 2.0 ** -10 * scale + 2.0 ** -20 * more
                assert np.all(np.abs(have - exact) <= bound)
        else:
            got = tuple(f64(p)[blk, :, off] for p in (self.cache.k_pool, self.cache.v_pool))
            _close(got[0], wk, size[:, HQ:], "bf16", "k")
            assert np.array_equal(got[1], wv)
        for i, r in enumerate(rows):
            assert len(self.k[r]) == slots[i]
            self.k[r].append(got[0][i])
            self.v[r].append(got[1][i])
        return q_out

    def attend(self, q, cu, shared, most, what):
        lens = [len(x) for x in self.k]
        call = self.kv.decode_shared_fp8 if self.fp8 else self.kv.decode_shared
        got = f64(call(self.cfg, self.cache, q, torch.from_numpy(self.table).cuda(), self.device(lens), max(lens),
                       self.device(cu), self.device(shared), most))
        assert self.kv.get_device_status() == 0
        for r, n in enumerate(lens):
            want, mag = attend(f64(q[r:r + 1]), np.array(self.k[r]), np.array(self.v[r]), np.ones((1, n), bool))
            check_attention(got[r:r + 1], want, mag, "bf16", f"{what}, sequence {r} of {n} tokens")

    def step(self, at, cu, shared, most, what):
        """A token for every sequence, then its attention; `at`: their next positions, moved on."""
        lens = [len(x) for x in self.k]
        pairs = [p for p in (self.alloc.prepare_append(row, BLOCK, n, n + 1) for row, n in zip(self.table, lens)) if p]
        if pairs:
            self.kv.copy_blocks(self.cfg, self.cache, *zip(*pairs))
        q = self.append(list(range(len(lens))), lens, [list(at)] * 3)
        at += 1
        self.attend(q, cu, shared, most, what)
        return len(pairs)


def _prompt(words, side, more):
    """Positions [3, T] of words, an image of side x side tokens, and more words."""
    t = [(i,) * 3 for i in range(words)]
    t += [(words, words + y, words + x) for y in range(side) for x in range(side)]
    t += [(words + side + i,) * 3 for i in range(more)]
    return np.array(t).T


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("once", [False, True])
def test_samples_of_image_prompts(kvattn_lib, kind, once):
    s = Server(kvattn_lib, kind, 8, 21)
    prompts, cu = [_prompt(70, 9, 11), _prompt(20, 14, 12)], [0, 5, 8]  # 162 tokens, and 228
    lens = [p.shape[1] for p in prompts]
    for first, n, p in zip(cu, lens, prompts):
        s.alloc.grow(s.table[first], BLOCK, 0, n)
        s.append([first] * n, list(range(n)), p.tolist())
    copies = 0
    for first, end, n in zip(cu, cu[1:], lens):
        for r in range(first + 1, end):
            s.alloc.fork(s.table[first], s.table[r], BLOCK, n)
            s.k[r], s.v[r] = list(s.k[first]), list(s.v[first])
    at = np.repeat([p.max() + 1 for p in prompts], np.diff(cu))
    most = LOOSE if once else max(lens)
    for i in range(21):
        copies += s.step(at, cu, lens, most, f"step {i}")
    assert copies == 4 + 2  # the blocks that the prompts end in; the last sample keeps the first's
    # evict some of the samples' own tokens: none, all, every other, the first ones, ...
    own = [list(range(lens[0], lens[0] + 21))] * 5 + [list(range(lens[1], lens[1] + 21))] * 3
    keep = [own[0], [], own[2][::2], own[3][5:], own[4][:3] + own[4][17:], own[5][1:2], own[6][:-1], own[7][4:9]]
    starts = [lens[0]] * 5 + [lens[1]] * 3
    cu_keep = np.cumsum([0] + [len(x) for x in keep])
    s.kv.compact_tokens(s.cfg, s.cache, torch.from_numpy(s.table).cuda(), s.device(starts), s.device(cu_keep.tolist()),
                        s.device([p for x in keep for p in x]))
    free = s.alloc.num_free
    for r, x in enumerate(keep):
        n = len(s.k[r])
        s.k[r], s.v[r] = ([rows[p] for p in list(range(starts[r])) + x] for rows in (s.k[r], s.v[r]))
        s.alloc.shrink(s.table[r], BLOCK, n, len(s.k[r]))
    assert s.alloc.num_free > free
    for i in range(4):  # slots go on behind what was kept, positions where they were
        s.step(at, cu, lens, most, f"step {i} after the eviction")
    for r in range(8):
        s.alloc.release(s.table[r], BLOCK, len(s.k[r]))
    assert s.alloc.num_free == NB - 3
