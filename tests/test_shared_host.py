"""CPU tests of the refusals of the shared-prefix, compaction and several-axes calls (nothing is launched: the pointers
are never read), and of the host calls beside them."""
import ctypes

import numpy as np
import pytest

FAKE = ctypes.c_void_p(0x7F0000001000)
ODD = ctypes.c_void_p(0x7F0000001008)


@pytest.fixture(scope="module")
def kv():
    import kv_cache_attention_rope_gb300 as kv

    return kv


def _code(kv, name):
    return kv.STATUS_CODE["KVATTN_" + name]


def _cache(kv, fp8, block=16, pool=FAKE):
    return kv.CacheFP8Desc(pool, 8, block) if fp8 else kv.CacheDesc(pool, pool, 8, block)


def _shared(kv, cfg=None, fp8=False, batch=0, max_len=64, cu=FAKE, shared=FAKE, groups=0, most=32, ws=FAKE, nbytes=1 << 40,
            q=FAKE, cache=None):
    cfg = cfg or kv.make_config(8, 2, 128, kv.BF16)
    cache = cache or _cache(kv, fp8)
    fn = kv.lib.kvattn_decode_shared_fp8 if fp8 else kv.lib.kvattn_decode_shared
    return fn(ctypes.byref(cfg), ctypes.byref(cache), q, FAKE, 4, FAKE, batch, max_len, cu, shared, groups, most, FAKE, ws,
              nbytes, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_shared_refusals(kv, fp8):
    ok, bad, uns = (_code(kv, n) for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED"))
    assert _shared(kv, fp8=fp8) == ok  # no sequences: nothing launched
    assert _shared(kv, fp8=fp8, cu=None, shared=None) == ok
    for more in (dict(batch=-1), dict(max_len=-1), dict(groups=-1), dict(most=-1), dict(batch=2, groups=3),
                 dict(batch=2, groups=1, cu=None), dict(batch=2, groups=1, shared=None), dict(batch=2, groups=1, q=None),
                 dict(batch=2, groups=1, q=ODD)):
        assert _shared(kv, fp8=fp8, **more) == bad, more
    assert _shared(kv, fp8=fp8, batch=9000) == uns
    assert _shared(kv, fp8=fp8, cfg=kv.make_config(9, 3, 128, kv.BF16)) == uns
    assert _shared(kv, fp8=fp8, cfg=kv.make_config(8, 2, 96, kv.BF16)) == uns
    small = _code(kv, "ERR_WORKSPACE_TOO_SMALL")
    assert _shared(kv, fp8=fp8, batch=2, groups=1, max_len=4000, most=3000, nbytes=64) == small
    assert _shared(kv, fp8=fp8, batch=2, groups=1, max_len=4000, most=3000, ws=None) == small


def test_decode_shared_fp8_only_refusals(kv):
    uns, bad = _code(kv, "ERR_UNSUPPORTED"), _code(kv, "ERR_INVALID_ARG")
    assert _shared(kv, fp8=True, cfg=kv.make_config(8, 4, 128, kv.BF16)) == uns   # groups of 2
    assert _shared(kv, fp8=True, cfg=kv.make_config(8, 2, 64, kv.BF16)) == uns
    assert _shared(kv, fp8=True, cfg=kv.make_config(8, 2, 128, kv.F32)) == uns
    assert _shared(kv, fp8=True, cache=kv.CacheFP8Desc(FAKE, 8, 24)) == bad


def test_decode_shared_workspace(kv):
    cfg = kv.make_config(32, 8, 128, kv.BF16)
    size = kv.decode_shared_workspace_size
    assert size(cfg, 4, 1000, 1, 500) > 0
    assert size(cfg, 0, 1000, 0, 0) >= 0
    assert size(cfg, -1, 1000, 0, 4) == size(cfg, 4, -5, 1, 4) == size(cfg, 4, 100, 5, 4) == size(cfg, 4, 100, -1, 4) == 0
    assert size(cfg, 4, 100, 1, -4) == size(kv.make_config(9, 3, 128, kv.BF16), 4, 100, 1, 4) == 0
    for i in range(4):
        args = [4, 1000, 1, 500]
        args[i] = 2 ** 32 + 1
        with pytest.raises(ValueError):
            size(cfg, *args)


def _compact(kv, kind="rows", cfg=None, starts=FAKE, cu=FAKE, keep=FAKE, total=0, table=FAKE, seqs=1, maxb=4, block=16,
             base=FAKE, layers=2, nblocks=8):
    cfg = cfg or kv.make_config(8, 2, 128, kv.BF16)
    lists = (starts, cu, keep, total, table, seqs, maxb, None)
    if kind == "layers":
        return kv.lib.kvattn_compact_tokens_layered(ctypes.byref(cfg), base, layers, nblocks, block, *lists)
    fn = kv.lib.kvattn_compact_tokens_fp8 if kind == "fp8" else kv.lib.kvattn_compact_tokens
    return fn(ctypes.byref(cfg), ctypes.byref(_cache(kv, kind == "fp8", block, base)), *lists)


@pytest.mark.parametrize("kind", ["rows", "fp8", "layers"])
def test_compact_refusals(kv, kind):
    ok, bad, uns = (_code(kv, n) for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED"))
    assert _compact(kv, kind) == ok                    # nothing kept: nothing launched
    assert _compact(kv, kind, total=5, seqs=0) == ok
    for more in (dict(total=-1), dict(seqs=-1), dict(maxb=0), dict(total=5, starts=None), dict(total=5, cu=None),
                 dict(total=5, keep=None), dict(total=5, table=None), dict(base=None), dict(base=ODD), dict(block=24),
                 dict(block=0)):
        assert _compact(kv, kind, **more) == bad, more
    assert _compact(kv, kind, cfg=kv.make_config(9, 3, 128, kv.BF16)) == uns
    assert _compact(kv, kind, cfg=kv.make_config(8, 2, 96, kv.BF16)) == uns
    assert _compact(kv, kind, cfg=kv.make_config(8, 2, 128, 7)) == bad
    if kind == "fp8":
        assert _compact(kv, kind, cfg=kv.make_config(8, 2, 64, kv.BF16)) == uns
        assert _compact(kv, kind, cfg=kv.make_config(8, 2, 128, kv.F32)) == uns
    if kind == "layers":
        assert _compact(kv, kind, layers=0) == bad and _compact(kv, kind, nblocks=0) == bad
        assert _compact(kv, kind, nblocks=2 ** 31) == bad
    fn = kv.lib.kvattn_compact_tokens
    assert fn(None, None, FAKE, FAKE, FAKE, 1, FAKE, 1, 1, None) == bad


def test_copy_blocks_fp8_refusals(kv):
    ok, bad, uns = (_code(kv, n) for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED"))

    def call(n=0, src=FAKE, dst=FAKE, cfg=None, block=16, pool=FAKE):
        return kv.lib.kvattn_copy_blocks_fp8(ctypes.byref(cfg or kv.make_config(8, 2, 128, kv.BF16)),
                                             ctypes.byref(kv.CacheFP8Desc(pool, 8, block)), src, dst, n, None)

    assert call() == ok
    for more in (dict(n=-1), dict(n=2, src=None), dict(n=2, dst=None), dict(block=24), dict(pool=None), dict(pool=ODD)):
        assert call(**more) == bad, more
    assert call(cfg=kv.make_config(8, 2, 64, kv.BF16)) == uns and call(cfg=kv.make_config(8, 2, 128, kv.F32)) == uns
    assert kv.lib.kvattn_copy_blocks_fp8(None, None, FAKE, FAKE, 0, None) == bad


def _axes(kv, axes, fp8=False, form=None, T=0, slots=FAKE, positions=FAKE, cfg=None):
    cfg = cfg or kv.make_config(8, 2, 128, kv.BF16)
    fn = kv.lib.kvattn_rotary_append_axes_fp8 if fp8 else kv.lib.kvattn_rotary_append_axes
    return fn(ctypes.byref(cfg), ctypes.byref(form or kv.make_rotary("half")), None if axes is None else ctypes.byref(axes),
              ctypes.byref(_cache(kv, fp8)), FAKE, 1536, FAKE, 1536, FAKE, 1536, None, positions, slots, FAKE, FAKE, 1, 1, T,
              None)


@pytest.mark.parametrize("fp8", [False, True])
def test_axes_refusals(kv, fp8):
    ok, bad, uns = (_code(kv, n) for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED"))
    a = kv.make_axes
    for good in (a([64]), a([16, 24, 24]), a([0, 0, 64]), a([0, 64]), a([16, 16, 16, 16]), a([24, 20, 20], "cyclic"),
                 a([22, 21, 21], "cyclic"), a([16, 16, 16, 16], "cyclic"), a([64, 0, 0], "cyclic"), a([64], "cyclic"),
                 a([32, 32], "cyclic")):
        assert _axes(kv, good, fp8) == ok, list(good.sections)
    for wrong in (None, a([63]), a([16, 24, 25]), a([-1, 65]), a([2 ** 31 - 1, 2 ** 31 - 1, 66]), a([31, 33], "cyclic"),
                  a([21, 22, 21], "cyclic"), a([20, 22, 22], "cyclic"), kv.RopeAxes(0, 0), kv.RopeAxes(5, 0),
                  kv.RopeAxes(1, 2, (ctypes.c_int32 * 4)(64))):
        assert _axes(kv, wrong, fp8) == bad, wrong and list(wrong.sections)
    assert _axes(kv, a([8, 8]), fp8, kv.make_rotary("half", 32)) == ok
    assert _axes(kv, a([8, 8]), fp8, kv.make_rotary("half", 64)) == bad
    assert _axes(kv, a([8, 8]), fp8, kv.make_rotary("half", 40)) == uns
    assert _axes(kv, a([64]), fp8, T=4, slots=None) == bad
    assert _axes(kv, a([64]), fp8, T=4, positions=None) == bad
    assert _axes(kv, a([64]), fp8, T=-1) == bad


def test_make_axes(kv):
    for wrong in ([], [1, 2, 3, 4, 5]):
        with pytest.raises(ValueError):
            kv.make_axes(wrong)
    with pytest.raises(ValueError):
        kv.make_axes([2 ** 31])
    with pytest.raises(KeyError):
        kv.make_axes([64], "woven")
    with pytest.raises(TypeError):
        kv.make_axes([32.0, 32])


@pytest.mark.parametrize("cur,new", [(0, 0), (40, 40), (40, 33), (40, 32), (40, 31), (40, 1), (40, 0), (48, 16)])
def test_table_shrink(kv, cur, new):
    alloc = kv.BlockAllocator(6)
    row, child = np.full(5, -1, np.int32), np.full(5, -1, np.int32)
    alloc.grow(row, 16, 0, cur)
    alloc.fork(row, child, 16, min(cur, 20))
    was, free = row.copy(), alloc.num_free
    alloc.shrink(row, 16, cur, new)
    have, need = (cur + 15) // 16, (new + 15) // 16
    assert list(row[:need]) == list(was[:need]) and np.all(row[need:] == -1)
    shared = min((min(cur, 20) + 15) // 16, have)
    assert alloc.num_free - free == sum(i >= shared for i in range(need, have))  # the child holds the shared ones
    assert all(alloc.refcount(int(b)) == 1 for b in child[need:shared])
    alloc.grow(row, 16, new, cur)
    assert np.all(row[:have] >= 0)
    alloc.close()


def test_table_shrink_refusals(kv):
    alloc = kv.BlockAllocator(6)
    row = np.full(4, -1, np.int32)
    alloc.grow(row, 16, 0, 40)
    was, free = row.copy(), alloc.num_free
    for args in ((16, 40, 41), (16, 40, -1), (0, 40, 10), (16, 100, 10), (16, 64, 10)):  # (the last names a block -1)
        with pytest.raises(kv.KvattnError):
            alloc.shrink(row, *args)
        assert list(row) == list(was) and alloc.num_free == free
    with pytest.raises(TypeError):
        alloc.shrink(row.astype(np.int64), 16, 40, 10)


def test_new_names_without_the_extension_module(kv):
    general = kv._General
    for name in ("decode_shared", "rotary_append_axes", "compact_tokens", "copy_blocks_fp8"):
        assert getattr(general, name)(1, 2, 3) is None
