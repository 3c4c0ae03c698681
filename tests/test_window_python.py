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
