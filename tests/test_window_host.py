"""CPU tests of the refusals of the rotary and windowed calls (nothing is launched: the pointers are never read)."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x7F0000001000)
ALL = 2 ** 31 - 1


@pytest.fixture(scope="module")
def kv():
    import kv_cache_attention_rope_gb300 as kv

    return kv


def _code(kv, name):
    return kv.STATUS_CODE["KVATTN_" + name]


def _rotary(kv, cfg=None, form=None, cache=None, fp8=False, T=0, strides=None, q=FAKE, nseq=1, maxb=1, q_out=None):
    cfg = cfg or kv.make_config(8, 2, 128, kv.BF16)
    form = form or kv.make_rotary("half")
    if cache is None:
        cache = kv.CacheFP8Desc(FAKE, 8, 16) if fp8 else kv.CacheDesc(FAKE, FAKE, 8, 16)
    qs, ks, vs = strides or (1536, 1536, 1536)
    fn = kv.lib.kvattn_rotary_append_fp8 if fp8 else kv.lib.kvattn_rotary_append
    return fn(ctypes.byref(cfg), ctypes.byref(form), ctypes.byref(cache), q, qs, FAKE, ks, FAKE, vs, q_out, FAKE, FAKE,
              FAKE, nseq, maxb, T, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_rotary_refusals(kv, fp8):
    ok, bad, uns = (_code(kv, n) for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED"))
    inf, nan = float("inf"), float("nan")
    form = kv.make_rotary
    assert _rotary(kv, fp8=fp8) == ok  # no tokens: nothing launched
    for f in (form("half", 64), form("adjacent", 16), form(scaling="linear", factor=1.0),
              form(scaling="base", factor=8.0), form(scaling="parts", factor=4.0, original_len=4096.0)):
        assert _rotary(kv, form=f, fp8=fp8) == ok
    for f in (kv.Rotary(2, 0, 0), kv.Rotary(-1, 0, 0), kv.Rotary(0, 0, 4), kv.Rotary(0, 0, -1), kv.Rotary(0, -16, 0),
              form(amplitude=-1.0), form(amplitude=nan), form(amplitude=inf), form(scaling="linear", factor=0.5),
              form(scaling="linear", factor=nan), form(scaling="base", factor=inf),
              form(scaling="parts", factor=2.0), form(scaling="parts", factor=2.0, original_len=nan),
              form(scaling="parts", factor=2.0, original_len=1024.0, low=4.0, high=4.0),
              form(scaling="parts", factor=2.0, original_len=1024.0, low=-1.0)):
        assert _rotary(kv, form=f, fp8=fp8) == bad
    for f in (form("half", 8), form("half", 72), form("half", 144)):
        assert _rotary(kv, form=f, fp8=fp8) == uns
    assert _rotary(kv, cfg=kv.make_config(8, 2, 128, kv.BF16, rope_base=0.5), fp8=fp8) == bad
    assert _rotary(kv, cfg=kv.make_config(8, 2, 96, kv.BF16), fp8=fp8) == uns
    assert _rotary(kv, cfg=kv.make_config(2 ** 21, 2 ** 18, 128, kv.BF16), fp8=fp8) == uns
    assert _rotary(kv, T=-1, fp8=fp8) == bad
    assert _rotary(kv, nseq=0, fp8=fp8) == bad
    assert _rotary(kv, maxb=0, fp8=fp8) == bad
    assert _rotary(kv, strides=(1020, 1536, 1536), fp8=fp8) == bad
    assert _rotary(kv, strides=(1536, 1540, 1536), fp8=fp8) == bad
    assert _rotary(kv, strides=(1536, 1536, 2 ** 62), T=4, fp8=fp8) == bad
    assert _rotary(kv, T=4, q=None, fp8=fp8) == bad
    assert _rotary(kv, T=4, q=ctypes.c_void_p(0x7F0000001008), fp8=fp8) == bad
    assert _rotary(kv, T=4, q_out=ctypes.c_void_p(0x7F0000001008), fp8=fp8) == bad


def test_rotary_fp8_only_refusals(kv):
    uns, bad = _code(kv, "ERR_UNSUPPORTED"), _code(kv, "ERR_INVALID_ARG")
    assert _rotary(kv, cfg=kv.make_config(8, 2, 128, kv.F32), fp8=True) == uns
    assert _rotary(kv, cfg=kv.make_config(8, 2, 64, kv.BF16), fp8=True) == uns
    assert _rotary(kv, cache=kv.CacheFP8Desc(FAKE, 8, 24), fp8=True) == bad


def test_make_rotary_names(kv):
    with pytest.raises(KeyError):
        kv.make_rotary("thirds")
    with pytest.raises(KeyError):
        kv.make_rotary(scaling="cubic")


def _decode(kv, cfg=None, fp8=False, window=16, sinks=0, batch=0, max_len=64, splits=0, ws=FAKE, nbytes=1 << 30, q=FAKE,
            cache=None):
    cfg = cfg or kv.make_config(8, 2, 128, kv.BF16)
    if cache is None:
        cache = kv.CacheFP8Desc(FAKE, 8, 16) if fp8 else kv.CacheDesc(FAKE, FAKE, 8, 16)
    fn = kv.lib.kvattn_decode_window_fp8 if fp8 else kv.lib.kvattn_decode_window
    return fn(ctypes.byref(cfg), ctypes.byref(cache), q, FAKE, 4, FAKE, batch, max_len, window, sinks, splits, FAKE, ws,
              nbytes, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_window_refusals(kv, fp8):
    ok, bad, uns = (_code(kv, n) for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED"))
    assert _decode(kv, fp8=fp8) == ok  # no sequences: nothing launched
    assert _decode(kv, fp8=fp8, window=ALL, sinks=ALL) == ok
    for more in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(batch=-1), dict(max_len=-1), dict(splits=-1),
                 dict(batch=2, q=None), dict(batch=2, q=ctypes.c_void_p(0x7F0000001008))):
        assert _decode(kv, fp8=fp8, **more) == bad
    assert _decode(kv, fp8=fp8, batch=9000) == uns
    assert _decode(kv, fp8=fp8, cfg=kv.make_config(9, 3, 128, kv.BF16)) == uns
    small = _code(kv, "ERR_WORKSPACE_TOO_SMALL")
    assert _decode(kv, fp8=fp8, batch=2, max_len=4000, window=1000, splits=4, nbytes=64) == small
    assert _decode(kv, fp8=fp8, batch=2, max_len=4000, window=1000, splits=4, ws=None) == small


def test_decode_window_fp8_only_refusals(kv):
    uns, bad = _code(kv, "ERR_UNSUPPORTED"), _code(kv, "ERR_INVALID_ARG")
    assert _decode(kv, fp8=True, cfg=kv.make_config(8, 4, 128, kv.BF16)) == uns   # groups of 2
    assert _decode(kv, fp8=True, cfg=kv.make_config(8, 2, 64, kv.BF16)) == uns
    assert _decode(kv, fp8=True, cfg=kv.make_config(8, 2, 128, kv.F32)) == uns
    assert _decode(kv, fp8=True, cache=kv.CacheFP8Desc(FAKE, 8, 24)) == bad


def test_decode_window_workspace(kv):
    """It goes by the keys that a query sees, not by the cache's length."""
    cfg = kv.make_config(32, 8, 128, kv.BF16)
    size = kv.decode_window_workspace_size
    assert size(cfg, 4, 100000, 100, 4, 1000) == size(cfg, 4, 200000, 100, 4, 1000)
    assert size(cfg, 4, 100000, 100, 4, 1000) < size(cfg, 4, 100000, 1000, 4, 1000)
    assert size(cfg, 4, 100000, ALL, ALL, 16) == kv.decode_workspace_size(cfg, 4, 100000, 16)
    assert size(cfg, 4, 1000, 0, 4) == size(cfg, 4, 1000, 16, -1) == size(cfg, -1, 1000, 16, 4) == 0
    assert size(cfg, 4, -5, 16, 4) == 0


def _prefill(kv, cfg=None, fp8=False, window=16, sinks=0, chunks=0, max_q=64, total=128, ws=FAKE, nbytes=1 << 40, q=FAKE,
             block=16):
    cfg = cfg or kv.make_config(8, 2, 128, kv.BF16)
    if fp8:
        cache = kv.CacheFP8Desc(FAKE, 8, block)
        return kv.lib.kvattn_prefill_window_fp8(ctypes.byref(cfg), ctypes.byref(cache), q, FAKE, FAKE, FAKE, 4, chunks,
                                                max_q, total, window, sinks, FAKE, ws, nbytes, None)
    cache = kv.CacheDesc(FAKE, FAKE, 8, block)
    return kv.lib.kvattn_prefill_window(ctypes.byref(cfg), ctypes.byref(cache), q, FAKE, FAKE, FAKE, 4, chunks, max_q,
                                        total, window, sinks, FAKE, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_window_refusals(kv, fp8):
    ok, bad, uns = (_code(kv, n) for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED"))
    assert _prefill(kv, fp8=fp8) == ok  # no chunks: nothing launched
    assert _prefill(kv, fp8=fp8, chunks=2, total=0) == ok
    assert _prefill(kv, fp8=fp8, chunks=2, max_q=0) == ok
    for more in (dict(window=0), dict(sinks=-1), dict(chunks=-1), dict(max_q=-1), dict(total=-1), dict(chunks=2, q=None),
                 dict(chunks=2, q=ctypes.c_void_p(0x7F0000001008))):
        assert _prefill(kv, fp8=fp8, **more) == bad
    assert _prefill(kv, fp8=fp8, cfg=kv.make_config(8, 2, 128, kv.F32)) == uns
    assert _prefill(kv, fp8=fp8, cfg=kv.make_config(8, 2, 96, kv.BF16)) == uns
    assert _prefill(kv, fp8=fp8, block=24) == bad  # a paged cache's blocks are multiples of 16


def test_prefill_window_fp8_workspace(kv):
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    size = kv.prefill_window_fp8_workspace_size
    n = size(cfg, 16, 4, 2, 64, 16, 0)
    assert n > 0
    assert _prefill(kv, fp8=True, chunks=2, nbytes=n - 1) == _code(kv, "ERR_WORKSPACE_TOO_SMALL")
    assert _prefill(kv, fp8=True, chunks=2, ws=None) == _code(kv, "ERR_INVALID_ARG")
    assert _prefill(kv, fp8=True, cfg=kv.make_config(8, 2, 64, kv.BF16)) == _code(kv, "ERR_UNSUPPORTED")
    # bounded by the row's blocks, and by what the chunks see when that is less
    assert size(cfg, 16, 100, 2, 64, ALL, ALL) == size(cfg, 16, 100, 2, 64, 1600, 0)
    assert size(cfg, 16, 10000, 2, 64, 16, 0) < size(cfg, 16, 10000, 2, 64, 1000, 0)
    for bad in ((24, 4, 2, 64, 16, 0), (16, 0, 2, 64, 16, 0), (16, 4, -1, 64, 16, 0), (16, 4, 2, -1, 16, 0),
                (16, 4, 2, 64, 0, 0), (16, 4, 2, 64, 16, -1)):
        assert size(cfg, *bad) == 0
    # every block that a chunk of max_q rows can see has room: rows at any prefix, sinks and window in blocks of 32
    for window in (1, 31, 32, 33, 100):
        for sinks in (0, 1, 32, 33):
            for q in (1, 2, 31, 65):
                room = (size(cfg, 32, 50, 1, q, window, sinks) - size(cfg, 32, 50, 1, 0, 1, 0)) // (2 * 2 * 32 * 256)
                most = 0
                for p in range(0, 300):
                    low = max(0, p - window + 1)
                    blocks = {k // 32 for k in range(low, p + q)} | {k // 32 for k in range(min(sinks, p + q))}
                    most = max(most, len(blocks))
                base = 1  # blocks of the subtracted size: a run of 0 keys
                assert room + base >= most, (window, sinks, q)
