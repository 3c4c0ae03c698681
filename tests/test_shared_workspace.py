"""CPU tests of what decode_shared asks of its workspace: what the form that the call takes needs, not more."""
import pytest


@pytest.fixture(scope="module")
def kv():
    import kv_cache_attention_rope_gb300 as kv

    return kv


def _alone(kv, cfg, batch, max_len):
    return kv.decode_window_workspace_size(cfg, batch, max_len, 2 ** 31 - 1)


@pytest.mark.parametrize("heads,batch,groups,most", [((12, 12, 64), 4, 1, 576), ((32, 8, 128), 4, 1, 1000), ((32, 32, 128), 8, 4, 100),
                                                     ((64, 8, 128), 2, 1, 2048), ((8, 1, 64), 2048, 192, 16)])
def test_small_calls(kv, heads, batch, groups, most):
    """Calls that read each sequence by itself, in both kinds of cache, ask for what that needs."""
    cfg = kv.make_config(*heads, kv.BF16)
    assert kv.decode_shared_workspace_size(cfg, batch, most + 64, groups, most) == _alone(kv, cfg, batch, most + 64)


@pytest.mark.parametrize("heads,batch,groups,most", [((32, 32, 128), 384, 192, 512), ((64, 8, 128), 400, 192, 1024),
                                                     ((32, 8, 128), 2048, 192, 4096), ((32, 8, 128), 64, 1, 2048)])
def test_states_of_real_rows(kv, heads, batch, groups, most):
    """Calls that read prefixes once: the states of the rows that there are, of a range of each SM besides, of own keys
    (at most 16 ranges an SM), and not of 256 rows for every group and KV head."""
    hq, hkv, d = heads
    cfg = kv.make_config(*heads, kv.BF16)
    got = kv.decode_shared_workspace_size(cfg, batch, most + 256, groups, most)
    sms = 160
    rows = sms * 256 + batch * hq + (sms * 16 + batch * hkv) * (hq // hkv)
    assert got <= max(_alone(kv, cfg, batch, most + 256), rows * (d + 2) * 4 + batch * 48 + 2048)
    assert got >= batch * hq * (d + 2) * 4


@pytest.mark.parametrize("heads", [(32, 8, 128), (12, 12, 64), (8, 1, 64)])
@pytest.mark.parametrize("bound", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 15])
def test_largest_bounds(kv, heads, bound):
    """A bound whose last page would end past 2^31 is one like any other."""
    cfg = kv.make_config(*heads, kv.BF16)
    near = 2 ** 31 - 16
    assert kv.decode_workspace_size(cfg, 2, bound) == kv.decode_workspace_size(cfg, 2, near) > 0
    assert _alone(kv, cfg, 2, bound) == _alone(kv, cfg, 2, near) > 0
    assert kv.decode_shared_workspace_size(cfg, 2, bound, 1, 1 << 20) == kv.decode_shared_workspace_size(cfg, 2, near, 1, 1 << 20)
