"""Caches whose sequences begin alike, and plain forms of token compaction, for the tests of the calls that share."""
from __future__ import annotations

import numpy as np
import torch

from oracle import fp8
from test_gpu_fp8 import _swz, pack_pages


class SharedCache:
    """groups: (shared tokens, lengths of the sequences).  The whole blocks of a group's common tokens are one copy, the
    block that they end in is a copy of each sequence's (as a fork and its first append leave them); a sequence no longer
    than the common tokens has the blocks of its length.  Slots that no sequence sees hold NaN, table entries without a
    seen token are -1 (all of a sequence of length 0)."""

    def __init__(self, kv, dtype, hkv, d, groups, block=16, seed=0, spare=3, own_rows=False):
        g = np.random.default_rng(seed)
        t = torch.bfloat16 if dtype != "f32" else torch.float32
        self.lens = [n for _, ls in groups for n in ls]
        self.cu = np.cumsum([0] + [len(ls) for _, ls in groups]).astype(np.int32)
        self.shared = np.array([s for s, _ in groups], np.int32)
        width = max(1, max((n + block - 1) // block for n in self.lens))
        self.k, self.v, cells, next_block = [], [], [], 0
        table = np.full((len(self.lens), width), -1, np.int64)
        rows_of = []  # (block, first token, tokens of the group's common part or own rows)
        for s, ls in groups:
            common = self._rows(g, dtype, s, hkv, d, t)
            whole = 0 if own_rows else s // block
            first = next_block
            next_block += whole
            used = max([min(n, s) for n in ls] + [0])
            for c in range(whole):
                rows_of.append((first + c, common, c * block, min(used, (c + 1) * block)))
            for n in ls:
                own = self._rows(g, dtype, max(0, n - s), hkv, d, t)
                seq = [np.concatenate([a[:min(n, s)], b]) for a, b in zip(common, own)]
                r = len(self.k)
                self.k.append(seq[0])
                self.v.append(seq[1])
                for c in range((n + block - 1) // block):
                    if c < whole:
                        table[r, c] = first + c
                    else:
                        table[r, c] = next_block
                        rows_of.append((next_block, seq, c * block, min(n, (c + 1) * block)))
                        next_block += 1
        nb = next_block + spare
        ids = g.permutation(nb)
        self.table = np.where(table >= 0, ids[table], -1).astype(np.int32)
        if dtype == "fp8":
            codes = np.full((2, nb, hkv, block, d), 0x7F, np.uint8)
            scales = np.full((2, nb, hkv, block), np.nan, np.float32)
        pools = np.full((2, nb, hkv, block, d), np.nan)
        for b, rows, a, e in rows_of:
            for i in range(2):
                if e <= a:
                    continue
                if dtype == "fp8":
                    codes[i][ids[b], :, :e - a], scales[i][ids[b], :, :e - a] = (
                        x.swapaxes(0, 1) for x in fp8.quantize_rows(rows[i][a:e]))
                else:
                    pools[i][ids[b], :, :e - a] = rows[i][a:e].swapaxes(0, 1)
        if dtype == "fp8":
            self.k, self.v = ([fp8.dequantize_rows(*fp8.quantize_rows(x)) if len(x) else x for x in xs]
                              for xs in (self.k, self.v))
            self.cache = kv.CacheFP8(torch.from_numpy(pack_pages(codes[0], scales[0], codes[1], scales[1])).cuda(), block)
        else:
            self.cache = kv.Cache(*(torch.from_numpy(p).to(t).cuda().contiguous() for p in pools))
        self.d_table, self.d_cu, self.d_shared = (torch.from_numpy(x).cuda() for x in (self.table, self.cu, self.shared))
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()

    @staticmethod
    def _rows(g, dtype, n, hkv, d, t):
        return list(torch.from_numpy(g.standard_normal((2, n, hkv, d))).to(t).double().numpy())


def compacted(pools, table, starts, lists, block):
    """numpy pools [..., blocks, hkv, block, D] after the move of each sequence's listed tokens to starts[s] ..."""
    out = pools.copy()
    for s, keep in enumerate(lists):
        for j, p in enumerate(keep):
            to = starts[s] + j
            out[..., table[s, to // block], :, to % block, :] = pools[..., table[s, p // block], :, p % block, :]
    return out


def _page_bytes(r):
    """Places in an fp8 page of token r's K codes, V codes, K scale and V scale."""
    lane = np.arange(128)
    k = r * 128 + ((lane // 16) ^ _swz(r)) * 16 + lane % 16
    return np.concatenate([k, 2048 + 16 * lane + r, 4096 + 4 * r + np.arange(4), 4160 + 4 * r + np.arange(4)])


def compacted_pages(pool, table, starts, lists, block):
    """The same of an fp8 pool [blocks, hkv, block // 16, 4224]."""
    out = pool.copy()
    for s, keep in enumerate(lists):
        for j, p in enumerate(keep):
            to = starts[s] + j
            src = pool[table[s, p // block], :, p % block // 16][:, _page_bytes(p % 16)]
            out[table[s, to // block], :, to % block // 16, _page_bytes(to % 16)] = src.T
    return out
