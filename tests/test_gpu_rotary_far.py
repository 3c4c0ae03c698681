"""GPU tests of rotary_append near the last position that an int32 names, against angles of 60 digits, and of forms used
in turn."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


def _pi():
    def atan_inverse(n):
        term, total, k = Decimal(1) / n, Decimal(1) / n, 1
        while abs(term) > Decimal(10) ** -62:
            term = -term / (n * n)
            k += 2
            total += term / k
        return total

    return 4 * (4 * atan_inverse(5) - atan_inverse(239))


def _speeds(base, rot, scaling, factor, original_len, low, high):
    """Speeds in turns per position, as kvattn.h states them, in 60 digits."""
    getcontext().prec = 60
    pi, b, s = _pi(), Decimal(base), Decimal(factor)
    if scaling == "base":
        b *= (s.ln() * Decimal(rot) / Decimal(rot - 2)).exp()
    out = []
    for i in range(rot // 2):
        f = (b.ln() * Decimal(-2 * i) / Decimal(rot)).exp()
        if scaling == "linear":
            f /= s
        elif scaling == "parts":
            g = min(Decimal(1), max(Decimal(0), (Decimal(original_len) * f / (2 * pi) - Decimal(low)) / Decimal(high - low)))
            f *= g + (1 - g) / s
        out.append(f / (2 * pi))
    return out


@pytest.mark.parametrize("base,scaling,factor", [(10000.0, "none", 1.0), (1e6, "none", 1.0), (500000.0, "parts", 8.0),
                                                 (10000.0, "linear", 1.5), (10000.0, "base", 4.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_far_positions(kvattn_lib, base, scaling, factor, d):
    """x = (1, 0) becomes (cos, sin) of the angle.  The angle's fraction of a turn is off by 2^31 half units of 2^-64
    turns, 2^-30 radians; its fp32 value by half a step of at most 1/4 half turns, pi / 4 * 2^-24 radians; sincospi by 1
    ulp of a value up to 1, 2^-24; the products are exact.  Together under 1.9 * 2^-24."""
    kv = kvattn_lib
    block = 2 ** 20
    T = 400
    pos = np.concatenate([TOP - np.arange(200), np.linspace(2 ** 30, TOP - 1000, T - 200).astype(np.int64)])
    cfg = kv.make_config(1, 1, d, kv.F32, rope_base=base)
    cache = kv.Cache(*(torch.zeros((1, 1, block, d), dtype=torch.float32, device="cuda") for _ in range(2)))
    table = torch.zeros((1, 2048), dtype=torch.int32, device="cuda")  # (their slots meet: the queries are looked at)
    q = torch.zeros((T, 1, d), dtype=torch.float32)
    q[..., :d // 2] = 1.0
    out = torch.empty((T, 1, d), dtype=torch.float32, device="cuda")
    low, high, original = 1.0, 32.0, 8192.0
    form = kv.make_rotary("half", 0, scaling, factor=factor, original_len=original, low=low, high=high)
    k = torch.zeros((T, 1, d), dtype=torch.float32, device="cuda")
    kv.rotary_append(cfg, form, cache, q.cuda(), k, k, torch.from_numpy(pos.astype(np.int32)).cuda(),
                     torch.zeros(T, dtype=torch.int32, device="cuda"), table, q_out=out)
    assert kv.get_device_status() == 0
    got = out.double().cpu().numpy()[:, 0]
    speeds = _speeds(base, d, scaling, factor, original, low, high)
    turns = np.array([[float((int(p) * f) % 1) for f in speeds] for p in pos])  # to 2^-53
    want = np.concatenate([np.cos(2 * np.pi * turns), np.sin(2 * np.pi * turns)], 1)
    worst = np.abs(got - want).max() * 2 ** 24
    assert worst < 1.9, worst


def test_forms_in_turn(kvattn_lib):
    """More rotary forms than a host thread keeps, in turn: each as when it is used alone."""
    kv = kvattn_lib
    T, d = 5, 128
    cache = kv.Cache(*(torch.zeros((4, 1, 16, d), dtype=torch.float32, device="cuda") for _ in range(2)))
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    q = torch.from_numpy(np.random.default_rng(0).standard_normal((T, 1, d))).float().cuda()
    pos = torch.arange(40, 40 + T, dtype=torch.int32, device="cuda")
    forms = [(kv.make_config(1, 1, d, kv.F32, rope_base=b), kv.make_rotary("half", r, s, factor=f))
             for b, r, s, f in ((1e4, 0, "none", 1.0), (1e6, 0, "none", 1.0), (1e4, 64, "none", 1.0), (1e4, 0, "linear", 2.0),
                                (1e4, 0, "linear", 4.0), (1e4, 0, "base", 4.0), (1e4, 16, "base", 4.0))]

    def run(cfg, form):
        out = torch.empty_like(q)
        kv.rotary_append(cfg, form, cache, q, q, q, pos, pos * 0, table, q_out=out)
        return out

    alone = [[run(*f) for _ in range(2)][1] for f in forms]
    for order in (range(7), reversed(range(7)), [0, 5, 0, 6, 1, 0, 2, 3, 4, 0, 5]):
        for i in order:
            assert torch.equal(run(*forms[i]), alone[i]), i
    assert len({x.cpu().numpy().tobytes() for x in alone}) == 7
