"""Plain 64-bit forms of the rotary append and of windowed attention, and cache builders for their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import fp8
from test_gpu_fp8 import pack_pages

TORCH_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # torch.finfo(t).eps / 2, relative


def speeds(base, rot, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        if scaling == "base":
            out.append((base * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot))
            continue
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            g = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
            f *= g + (1 - g) / factor
        out.append(f)
    return np.array(out)


def rotate(x, positions, f, rot, layout, amplitude):
    """x [T, H, D] in 64 bits: its rotation, and |x0| + |x1| of each element's pair (0 where copied)."""
    x = np.asarray(x, np.float64)
    y, size = x.copy(), np.zeros_like(x)
    a = np.asarray(positions, np.float64)[:, None] * f
    c, s = (np.cos(a) * amplitude)[:, None], (np.sin(a) * amplitude)[:, None]
    n = rot // 2
    i0 = np.arange(n) if layout == "half" else 2 * np.arange(n)
    i1 = i0 + (n if layout == "half" else 1)
    x0, x1 = x[..., i0], x[..., i1]
    y[..., i0] = x0 * c - x1 * s
    y[..., i1] = x0 * s + x1 * c
    size[..., i0] = size[..., i1] = amplitude * (np.abs(x0) + np.abs(x1))
    return y, size


def seen(pos, n, window, sinks):
    """[len(pos), n]: the row at position pos[r] sees key j."""
    j = np.arange(n)[None, :]
    p = np.asarray(pos, np.int64)[:, None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def attend(q, k, v, mask):
    """q [R, Hq, D], k and v [n, Hkv, D], mask [R, n] in 64 bits: the output and sum of weight * |v|; keys that a row
    does not see may hold anything."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    R, hq, d = q.shape
    hkv = k.shape[1]
    out, mag = np.zeros((R, hq, d)), np.zeros((R, hq, d))
    for r in range(R):
        idx = np.nonzero(mask[r])[0]
        if not len(idx):
            continue
        kk, vv = k[idx], v[idx]
        for h in range(hkv):
            g = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            s = q[r, g] @ kk[:, h].T / math.sqrt(d)
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[r, g], mag[r, g] = w @ vv[:, h], w @ np.abs(vv[:, h])
    return out, mag


def check_attention(got, want, mag, dtype, what):
    """|got - want| within the roundings.  bf16: each weight is rounded to bf16 before P.V (half a step, 2^-8 relative,
    of each w |v|) and the output once (2^-8 |out|); the fp32 score sums (128 products of up to ~16 in all: 128 *
    2^-24 * 16 = 2^-13 absolute, so 2^-12 relative on a weight after its normalisation) and exp2 add less than 2^-11.
    fp8: the weights are rounded to f16 (2^-11), as are V and K in a prefill: 2^-11 for V, and for K errors of up to
    2^-11 |q k| in each of 128 products, independent, so 2^-11 / sqrt(3) of sqrt(sum (q k)^2 / 128), which is about 1: six
    standard deviations are 2^-9.2 of a score, and of a weight.  f32: the scores' and the output's alone."""
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    weight = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -10 + 2.0 ** -9, "f32": 0.0}[dtype] + 2.0 ** -11
    bound = weight * mag + HALF_STEP["f32" if dtype == "f32" else "bf16"] * (np.abs(want) + weight * mag) + 1e-30
    over = np.abs(got - want) - bound
    assert np.all(over <= 0), f"{what}: {over.max():.3e} past the bound"
    if dtype == "f32" and want.size:  # the errors of the sums are random: far under their bound together
        assert np.linalg.norm(got - want) <= 1e-5 * max(np.linalg.norm(want), 1e-30), what


class WindowCache:
    """Sequences of the given lengths in a cache whose every slot that `wanted[r]` (a boolean per token) does not name
    holds NaN, and whose table has -1 for blocks without a named token."""

    def __init__(self, kv, dtype, hkv, d, lens, wanted, block=16, seed=0, spare=3):
        g = np.random.default_rng(seed)
        self.dtype, n = dtype, len(lens)
        width = max(1, max((L + block - 1) // block for L in lens))
        cells = [(r, c) for r, L in enumerate(lens) for c in range((L + block - 1) // block)
                 if wanted[r][c * block:(c + 1) * block].any()]
        nb = len(cells) + spare
        ids = g.permutation(nb)
        self.table = np.full((n, width), -1, np.int32)
        self.k, self.v = [], []
        pools = np.full((2, nb, hkv, block, d), np.nan)
        for (r, c), b in zip(cells, ids):
            self.table[r, c] = b
        t = torch.bfloat16 if dtype != "f32" else torch.float32
        codes = np.full((2, nb, hkv, block, d), 0x7F, np.uint8)          # e4m3 NaN
        scales = np.full((2, nb, hkv, block), np.nan, np.float32)
        for r, L in enumerate(lens):
            rows = torch.from_numpy(g.standard_normal((2, L, hkv, d))).to(t).double().numpy()
            tok = np.nonzero(wanted[r][:L])[0]
            at = (self.table[r, tok // block], slice(None), tok % block)
            if dtype == "fp8":
                for i in range(2):
                    c, s = fp8.quantize_rows(rows[i])
                    codes[i][at], scales[i][at] = c[tok], s[tok]
                    rows[i] = fp8.dequantize_rows(c, s)
            for i in range(2):
                pools[i][at] = rows[i][tok]
            self.k.append(rows[0])
            self.v.append(rows[1])
        if dtype == "fp8":
            self.cache = kv.CacheFP8(torch.from_numpy(pack_pages(codes[0], scales[0], codes[1], scales[1])).cuda(), block)
        else:
            self.cache = kv.Cache(*(torch.from_numpy(p).to(t).cuda().contiguous() for p in pools))
        self.d_table = torch.from_numpy(self.table).cuda()
