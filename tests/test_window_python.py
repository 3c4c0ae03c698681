"""CPU tests of the Python side of the rotary and windowed calls."""
import pytest


@pytest.fixture(scope="module")
def kv():
    import kv_cache_attention_rope_gb300 as kv

    return kv


def test_sizes_past_32_bits(kv):
    """An integer that does not fit 32 bits raises; its low 32 bits are not taken for it."""
    cfg = kv.make_config(8, 2, 128, kv.BF16)
    assert kv.decode_window_workspace_size(cfg, 4, 1000, 100, 4) > 0
    assert kv.prefill_window_fp8_workspace_size(cfg, 16, 64, 2, 50, 128, 4) > 0
    for wrong in (2 ** 32 + 16, 2 ** 31, -2 ** 32 + 16):
        for i in range(5):
            args = [4, 1000, 100, 4, 0]
            args[i] = wrong
            with pytest.raises(ValueError):
                kv.decode_window_workspace_size(cfg, *args)
        for i in range(6):
            args = [16, 64, 2, 50, 128, 4]
            args[i] = wrong
            with pytest.raises(ValueError):
                kv.prefill_window_fp8_workspace_size(cfg, *args)
        with pytest.raises(ValueError):
            kv.make_rotary("half", wrong)
    with pytest.raises(TypeError):
        kv.make_rotary("half", 64.0)


def test_package_without_the_extension_module():
    """Where the extension module is not built, or is another Python's, the package is all there."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import sys
sys.modules['kv_cache_attention_rope_gb300._marshal'] = None     # importing it raises ImportError
import kv_cache_attention_rope_gb300 as kv
assert kv._marshal.decode_window(1, 2) is None
cfg = kv.make_config(8, 2, 128, kv.BF16)
assert kv.version() > 0 and kv.decode_window_workspace_size(cfg, 4, 1000, 100) > 0
alloc = kv.BlockAllocator(4)
assert len(alloc.alloc(3)) == 3
print('whole')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "whole" in r.stdout, r.stderr


def test_extension_module_is_built_for_one_python(kv, tmp_path, monkeypatch):
    """Its file name has the Python's tag, and without Python's headers the build goes without it."""
    import importlib.machinery
    import os
    import sysconfig

    build = kv._build
    assert any("cpython" in s and build.MARSHAL.endswith("_marshal" + s) for s in importlib.machinery.EXTENSION_SUFFIXES)
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / os.path.basename(build.MARSHAL)))
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    build._build_marshal(True, [])
    assert not os.listdir(tmp_path)


def test_rotary_fp8_refuses_more_kv_heads_than_its_grid_holds(kv):
    """Before anything is launched: K and q would have been stored, and V not."""
    import ctypes

    fake = ctypes.c_void_p(0x7F0000001000)

    def call(hkv, fp8):
        cfg, form = kv.make_config(hkv, hkv, 128, kv.BF16), kv.make_rotary("half")
        cache = kv.CacheFP8Desc(fake, 8, 16) if fp8 else kv.CacheDesc(fake, fake, 8, 16)
        row = 128 * hkv
        fn = kv.lib.kvattn_rotary_append_fp8 if fp8 else kv.lib.kvattn_rotary_append
        return fn(ctypes.byref(cfg), ctypes.byref(form), ctypes.byref(cache), fake, row, fake, row, fake, row, None, fake, fake,
                  fake, 1, 1, 0, None)

    ok, uns = kv.STATUS_CODE["KVATTN_OK"], kv.STATUS_CODE["KVATTN_ERR_UNSUPPORTED"]
    assert call(65535, True) == ok and call(65536, True) == uns
    assert call(2 ** 20, False) == ok and call(2 ** 20 + 1, False) == uns
